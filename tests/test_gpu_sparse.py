"""sage_attn_fwd_sparse: attention over listed key blocks, in every mode.

Against the formula in 64 bits, element by element.  Derived bounds (half steps: bf16 2^-8, fp32 2^-24):
BF16: each p is rounded to bf16 (2^-8 of p), the result once more; a score is a product of d terms summed in
  fp32, off by at most (d + 8) * 2^-24 * sum |q||k| / sqrt(d), which moves p by that much (twice: in p and in
  the row sum); exponentials, sums and rescalings add under 2^-16.
INT8/FP8: codes and integer scores are exact; s and m are rounded in fp32, so p is known to
  eta = 2^-21 * (largest |s| + 16): a P8 code may fall on either side of a rounding border that lies within
  eta, which costs the difference of the two codes; everything else adds under 2^-16 + eta of sum p|v| / l.
And bit by bit: a list of all blocks in order is the dense call.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, I8, QTOK = 0, 1, 2
MODES = [BF16, I8, QTOK]


def bits(t):
    return t.view(torch.int16)


def inputs(B, H, N, d, seed, dev, off=3.0):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    q, k, v = (torch.randn((B, H, N, d), generator=g, device=dev) for _ in range(3))
    k += off * torch.randn((B, H, 1, d), generator=g, device=dev)
    return tuple(t.to(torch.bfloat16) for t in (q, k, v)) + (g,)


def random_lists(B, H, nT, width, g, dev, lo=0):
    """Distinct blocks in no order, lo .. min(width, nT) of them, -1 behind."""
    G = B * H * nT
    order = torch.rand((G, nT), generator=g, device=dev).argsort(dim=1)
    n = min(width, nT)
    lists = torch.full((G, width), -1, dtype=torch.int32, device=dev)
    lists[:, :n] = order[:, :n].to(torch.int32)
    counts = torch.randint(lo, n + 1, (G,), generator=g, device=dev).to(torch.int32)
    lists[torch.arange(width, device=dev)[None] >= counts[:, None]] = -1
    return lists.view(B, H, nT, width).contiguous(), counts.view(B, H, nT).contiguous()


def all_blocks(B, H, nT, dev):
    return (torch.arange(nT, dtype=torch.int32, device=dev).expand(B, H, nT, nT).contiguous(),
            torch.full((B, H, nT), nT, dtype=torch.int32, device=dev))


def e4m3(x):
    return x.float().clamp(-448, 448).to(torch.float8_e4m3fn).double()


def expect(q, k, v, mode, lists, counts):
    """(value, allowed error) in fp64 for each element."""
    from video_dit_quantized_b200 import sage
    B, H, N, d = q.shape
    nT = -(-N // 128)
    val = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(val)
    pre = sage.quantize_qk(q, k, v, q_per_token=mode == QTOK) if mode != BF16 else None
    LL, CC = lists.cpu().tolist(), counts.cpu().tolist()
    for b in range(B):
        for h in range(H):
            for i in range(nT):
                L = LL[b][h][i][:CC[b][h][i]]
                if not L:
                    continue
                r = slice(i * 128, min(N, i * 128 + 128))
                spans = [slice(j * 128, min(N, j * 128 + 128)) for j in L]
                if mode == BF16:
                    kk = torch.cat([k[b, h, s] for s in spans]).double()
                    vv = torch.cat([v[b, h, s] for s in spans]).double()
                    qq = q[b, h, r].double()
                    s = qq @ kk.T / math.sqrt(d)
                    eps = (d + 8) * 2.0 ** -24 * (qq.abs() @ kk.abs().T / math.sqrt(d)).amax(1, keepdim=True)
                    p = torch.softmax(s, dim=1)
                    o = p @ vv
                    val[b, h, r] = o
                    tol[b, h, r] = 2 ** -8 * o.abs() + (2 ** -8 + 2 * eps + 2 ** -16) * (p @ vv.abs()) * 1.01
                    continue
                rows = r.stop - r.start
                qi = pre["q_i8"][b, h, r].double()
                sc = (pre["q_scale"][b, h, r][:, None] if mode == QTOK else pre["q_scale"][b, h, i]).double()
                m = torch.full((rows, 1), -math.inf, dtype=torch.float64, device=q.device)
                l, acc, slack, mass = (torch.zeros((rows, n), dtype=torch.float64, device=q.device) for n in (1, d, d, d))
                vs = pre["v_scale"][b, h].double()
                for j, sp in zip(L, spans):
                    ks = pre["k_scale"][b, h, j].double()
                    s = (qi @ pre["k_i8"][b, h, sp].double().T) * sc * ks * (math.log2(math.e) / math.sqrt(d))
                    v8 = pre["v_f8t"][b, h][:, sp].view(torch.float8_e4m3fn).double().T
                    m2 = torch.maximum(m, s.amax(1, keepdim=True))
                    a, p = torch.exp2(m - m2), torch.exp2(s - m2)
                    eta = 2.0 ** -21 * (s.abs().amax() + m2.abs().amax() + 16)
                    step = e4m3(p * 448 * (1 + eta)) - e4m3(p * 448 * (1 - eta))
                    l = l * a + p.sum(1, keepdim=True)
                    acc = acc * a + e4m3(p * 448) @ v8
                    slack = slack * a + (step + p * 448 * (2 ** -16 + 2 * eta)) @ v8.abs()
                    m = m2
                o = acc * vs / (448 * l)
                val[b, h, r] = o
                tol[b, h, r] = 2 ** -8 * o.abs() + 1.01 * slack * vs / (448 * l)
    return val, tol


def check(q, k, v, mode, lists, counts, seed_ws=None):
    from video_dit_quantized_b200 import sage, sparse
    B, H, N, d = q.shape
    ws = sage.alloc_workspace(B, H, N, d, mode, q.device)
    pad = torch.full((q.numel() + 512,), 9.0, dtype=torch.bfloat16, device=q.device)
    o = pad[256:256 + q.numel()].view(q.shape)
    sparse.attn_fwd_sparse(q, k, v, mode, lists, counts, o=o, workspace=ws)
    assert sage.status(ws) == sage.OK
    val, tol = expect(q, k, v, mode, lists, counts)
    err = (o.double() - val).abs()
    assert torch.isfinite(o).all()
    assert (err <= tol).all(), (float((err - tol).max()), int((err > tol).sum()))
    assert (pad[:256] == 9).all() and (pad[256 + q.numel():] == 9).all()
    empty = (counts == 0)[..., None].expand(-1, -1, -1, 128).reshape(B, H, -1)[:, :, :N]
    assert (o[empty] == 0).all()
    return o


SHAPES = [(1, 1, 1, 128, 1), (1, 2, 127, 64, 1), (2, 1, 129, 128, 2), (1, 3, 300, 64, 5), (2, 2, 1000, 128, 4),
          (1, 2, 1000, 64, 8), (1, 1, 1700, 128, 14), (1, 2, 2500, 64, 7)]


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_ragged_lists_against_the_formula(shape, mode, cuda_dev):
    B, H, N, d, width = shape
    q, k, v, g = inputs(B, H, N, d, 100 + N + mode, cuda_dev)
    lists, counts = random_lists(B, H, -(-N // 128), width, g, cuda_dev)
    check(q, k, v, mode, lists, counts)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("B,H,N,d", [(1, 1, 1, 64), (2, 3, 385, 64), (1, 2, 1024, 128), (1, 3, 1500, 128), (1, 1, 4000, 64)])
def test_all_blocks_in_order_is_the_dense_call(B, H, N, d, mode, cuda_dev):
    from video_dit_quantized_b200 import sage, sparse
    q, k, v, _ = inputs(B, H, N, d, 7 + N, cuda_dev)
    lists, counts = all_blocks(B, H, -(-N // 128), cuda_dev)
    got = sparse.attn_fwd_sparse(q, k, v, mode, lists, counts)
    assert torch.equal(bits(got), bits(sage.attn_fwd(q, k, v, mode)))


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("c0,c1", [(0, 0), (0, 9), (9, 0), (1, 9), (9, 1), (2, 3), (3, 2), (9, 9), (4, 0), (5, 6)])
def test_neighbours_of_any_two_lengths(c0, c1, mode, cuda_dev):
    """The two query blocks of a CTA with lists of different lengths: same rows as alone, and right."""
    q, k, v, g = inputs(1, 1, 1100, 128, 3 * c0 + c1, cuda_dev)
    nT = 9
    lists, counts = random_lists(1, 1, nT, 9, g, cuda_dev, lo=9)
    n = torch.tensor([c0, c1] * 5, device=cuda_dev, dtype=torch.int32)[:nT]
    counts = n.view(1, 1, nT).contiguous()
    check(q, k, v, mode, lists, counts)


@pytest.mark.parametrize("mode", MODES)
def test_order_repeats_and_width(mode, cuda_dev):
    from video_dit_quantized_b200 import sparse
    q, k, v, g = inputs(1, 2, 900, 64, 40, cuda_dev)
    lists, counts = random_lists(1, 2, 8, 6, g, cuda_dev, lo=2)
    o = check(q, k, v, mode, lists, counts)
    wide = torch.full((1, 2, 8, 11), 77, dtype=torch.int32, device=cuda_dev)     # behind the counts: never read as blocks
    wide[..., :6] = lists
    assert torch.equal(bits(o), bits(sparse.attn_fwd_sparse(q, k, v, mode, wide, counts)))
    lists[..., 1] = lists[..., 0]                                               # a block twice
    check(q, k, v, mode, lists, counts)


@pytest.mark.parametrize("mode", MODES)
def test_bad_indices_and_counts_are_reported_and_skipped(mode, cuda_dev):
    """Runs after the index guards of the kernel: the load falls back to block 0, the scores are masked."""
    from video_dit_quantized_b200 import sage, sparse
    q, k, v, g = inputs(1, 2, 700, 128, 50, cuda_dev)
    lists, counts = random_lists(1, 2, 6, 4, g, cuda_dev, lo=3)
    ref = sparse.attn_fwd_sparse(q, k, v, mode, lists[..., :3].contiguous(), counts.clamp(max=3))
    ws = sage.alloc_workspace(1, 2, 700, 128, mode, cuda_dev)
    for bad in (-1, 6, 2 ** 31 - 1, -2 ** 31):
        for at in (0, 3):
            li = lists.clone()
            li[..., at] = bad
            if at == 0:
                li[..., 1:4] = lists[..., :3]
            got = sparse.attn_fwd_sparse(q, k, v, mode, li, (counts.clamp(max=3) + 1).contiguous(), workspace=ws)
            assert sage.status(ws) == sage.EINVAL
            assert sage.status(ws) == sage.OK
            assert torch.equal(bits(got), bits(ref)), (bad, at)
    only = torch.full_like(lists, 99)
    got = sparse.attn_fwd_sparse(q, k, v, mode, only, counts, workspace=ws)
    assert sage.status(ws) == sage.EINVAL and (got == 0).all()
    for c in (-5, 5, 2 ** 31 - 1):
        cc = counts.clone()
        cc[0, 1, 2] = c
        got = sparse.attn_fwd_sparse(q, k, v, mode, torch.where(lists < 0, 0, lists), cc, workspace=ws)
        assert sage.status(ws) == sage.EINVAL and torch.isfinite(got).all()
    # and the next call is clean
    again = sparse.attn_fwd_sparse(q, k, v, mode, lists[..., :3].contiguous(), counts.clamp(max=3), workspace=ws)
    assert sage.status(ws) == sage.OK and torch.equal(bits(again), bits(ref))


@pytest.mark.parametrize("mode", [I8, QTOK])
@pytest.mark.parametrize("d", [64, 128])
def test_reciprocal_coefficients_are_torch_codes(mode, d, cuda_dev):
    """COEFF_RECIPROCAL: the workspace holds the codes and scales of torch's `127.0 / amax` and `amax / 127.0` on the
    GPU, bit for bit; COEFF_DIVIDE holds those of sage_quantize_qk."""
    from video_dit_quantized_b200 import sage, sparse
    B, H, N = 1, 3, 3000
    nT, G = 24, 3
    q, k, v, g = inputs(B, H, N, d, 70, cuda_dev)
    v[0, 1, :, 3] = 0
    k[0, 2] = k[0, 2, :1]                                             # smoothed to zero: scale 0
    lists, counts = random_lists(B, H, nT, 3, g, cuda_dev, lo=1)
    size = {"q_i8": G * nT * 128 * d, "k_i8": G * nT * 128 * d, "v_f8t": G * nT * 128 * d,
            "q_scale": 4 * G * (nT * 128 if mode == QTOK else nT), "k_scale": 4 * G * nT, "k_mean": 4 * G * d,
            "v_scale": 4 * G * d}
    pad = lambda x: torch.nn.functional.pad(x.float().view(G, N, d), (0, 0, 0, nT * 128 - N)).view(G, nT, 128, d)
    mean = (k.double().sum(2, keepdim=True) / torch.full((), N, dtype=torch.float64, device=cuda_dev)).float()
    vmax = v.float().abs().amax(2).view(G, d)
    want = {"k_mean": mean.flatten(), "v_scale": (vmax / 448.0).flatten()}
    inv = torch.where(vmax > 0, 448.0 / vmax, 0.0)
    want["v_f8t"] = (pad(v) * inv[:, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).view(
        G, nT * 128, d).transpose(1, 2).flatten()
    for name, x, dims in (("q", pad(q), (3,) if mode == QTOK else (2, 3)), ("k", pad(k.float() - mean), (2, 3))):
        if name == "k":
            x[:, -1, N - (nT - 1) * 128:] = 0
        amax = x.abs().amax(dims, keepdim=True)
        want[name + "_scale"] = (amax / 127.0).flatten()
        want[name + "_i8"] = (x * torch.where(amax > 0, 127.0 / amax, 0.0)).round().clamp(-127, 127).to(torch.int8).flatten()
    for coeff in (sparse.COEFF_RECIPROCAL, sparse.COEFF_DIVIDE):
        ws = sage.alloc_workspace(B, H, N, d, mode, cuda_dev)
        sparse.attn_fwd_sparse(q, k, v, mode, lists, counts, coeff=coeff, workspace=ws)
        if coeff == sparse.COEFF_DIVIDE:
            pre = sage.quantize_qk(q, k, v, q_per_token=mode == QTOK)
            want = {n: pre[n].flatten() for n in size}
        at = 256
        for name, n in size.items():
            got = ws[at:at + n]
            assert torch.equal(got, want[name].contiguous().view(torch.uint8)), (name, coeff)
            at += -(-n // 256) * 256


def test_blocks_that_are_not_listed_are_not_touched(cuda_dev):
    """BF16: NaN and infinity in keys and values of other blocks change nothing (no statistics cross blocks)."""
    from video_dit_quantized_b200 import sparse
    q, k, v, g = inputs(1, 1, 1000, 128, 60, cuda_dev)
    lists = torch.tensor([1, 2, 7], dtype=torch.int32, device=cuda_dev).expand(1, 1, 8, 3).contiguous()
    counts = torch.full((1, 1, 8), 3, dtype=torch.int32, device=cuda_dev)
    ref = sparse.attn_fwd_sparse(q, k, v, BF16, lists, counts)
    for j, x in ((0, float("nan")), (3, float("inf")), (6, -float("inf"))):
        k[0, 0, j * 128:(j + 1) * 128] = x
        v[0, 0, j * 128:(j + 1) * 128] = x
    assert torch.equal(bits(ref), bits(sparse.attn_fwd_sparse(q, k, v, BF16, lists, counts)))


def test_forced_timeout_reports_and_recovers(cuda_dev):
    from video_dit_quantized_b200 import sage, sparse
    q, k, v, g = inputs(1, 2, 1024, 128, 61, cuda_dev)
    lists, counts = all_blocks(1, 2, 8, cuda_dev)
    for mode in MODES:
        ws = sage.alloc_workspace(1, 2, 1024, 128, mode, cuda_dev)
        sparse.dbg_sparse_forced_timeout(q, k, v, mode, lists, counts, ws, 20_000_000)
        assert sage.status(ws) == sage.ETIMEOUT
        o = sparse.attn_fwd_sparse(q, k, v, mode, lists, counts, workspace=ws)
        assert sage.status(ws) == sage.OK
        assert torch.equal(bits(o), bits(sage.attn_fwd(q, k, v, mode)))
