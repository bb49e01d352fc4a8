"""The sparse path as it is used: projections -> norm and rotation -> block choice -> attention, in one run; captured
into a graph; on other streams; through the debug build; and inside the Ulysses exchange."""
import contextlib
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, I8, QTOK = 0, 1, 2


def bits(t):
    return t.view(torch.int16) if t.dtype == torch.bfloat16 else t


def projections(B, N, H, d, seed, dev):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    qkv = torch.randn((B, N, 3, H, d), generator=g, device=dev)
    nT = -(-N // 128)
    slow = torch.randn((B, nT, 3, H, d), generator=g, device=dev)
    qkv = (qkv + slow.repeat_interleave(128, dim=1)[:, :N]).to(torch.bfloat16)
    w = [(1 + 0.1 * torch.randn(H * d, generator=g, device=dev)).to(torch.bfloat16) for _ in range(2)]
    a = torch.rand((N, d // 2), generator=g, device=dev, dtype=torch.float64) * 50
    return qkv, w, a.cos().float(), a.sin().float()


def layer(qkv, w, cos, sin, mode, keep, **kw):
    from video_dit_quantized_b200 import sparse
    q, k = sparse.qk_norm_rope(qkv[:, :, 0], qkv[:, :, 1], wq=w[0], wk=w[1], norm=sparse.NORM_RMS,
                               scope=sparse.NORM_SCOPE_ALL, cos=cos, sin=sin, **kw)
    v = qkv[:, :, 2].permute(0, 2, 1, 3).contiguous()
    lists, counts = sparse.select_blocks(q, k, keep, first=1, window=1, **kw)
    return q, k, v, lists, counts, sparse.attn_fwd_sparse(q, k, v, mode, lists, counts, **kw)


@pytest.mark.parametrize("mode", [BF16, I8, QTOK])
@pytest.mark.parametrize("B,N,H,d", [(1, 1300, 4, 128), (2, 777, 3, 64)])
def test_the_run_against_float64(B, N, H, d, mode, cuda_dev):
    """The three calls in a row against the same layer in 64 bits from the bf16 projections.  Every stage is tested
    to its own bound elsewhere; end to end, the BF16 rounding of q and k (2^-8 each, as a norm over d terms at
    random) moves scores of size ~ |q||k|/sqrt(d) = sqrt(d) by about 2^-8 and p with them: a few 2^-8 of |o| in
    norm.  INT8 codes (half a step of amax / 127, amax ~ 4 sigma: 1.6% of sigma, q and k at random) move scores by
    about 0.02 * sqrt(2), P8 and V8 (2^-4 of each value, at random, 0.6 of that in norm) add 2 * 3.6%."""
    from video_dit_quantized_b200 import sage, sparse
    qkv, w, cos, sin = projections(B, N, H, d, 3, cuda_dev)
    nT = -(-N // 128)
    q, k, v, lists, counts, o = layer(qkv, w, cos, sin, mode, 4)
    x = qkv.double()
    out = []
    for t in range(2):
        y = x[:, :, t]
        y = y / (y.square().mean((2, 3), keepdim=True) + 1e-6).sqrt() * w[t].double().view(H, d)
        a, b = y[..., 0::2], y[..., 1::2]
        co, si = cos.double()[None, :, None], sin.double()[None, :, None]
        out.append(torch.stack((a * co - b * si, a * si + b * co), -1).flatten(-2).permute(0, 2, 1, 3))
    mask = torch.zeros((B, H, nT, nT), dtype=torch.bool, device=cuda_dev)
    mask.scatter_(3, lists.long().clamp(min=0), lists >= 0)
    i = torch.arange(nT, device=cuda_dev)
    assert mask[..., 0].all() and mask[:, :, i, i].all() and (counts == 4).all()
    full = mask.repeat_interleave(128, 2).repeat_interleave(128, 3)[:, :, :N, :N]
    s = (out[0] @ out[1].transpose(-1, -2) / math.sqrt(d)).masked_fill(~full, -math.inf)
    ref = torch.softmax(s, -1) @ x[:, :, 2].permute(0, 2, 1, 3)
    rel = float((o.double() - ref).norm() / ref.norm())
    assert rel <= (0.02 if mode == BF16 else 0.12), rel


@pytest.mark.parametrize("mode", [BF16, I8, QTOK])
def test_replay_from_graphs(mode, cuda_dev):
    """Captured once, replayed on new inputs; two graphs share the workspace one after the other; an eager call
    between them changes nothing."""
    from video_dit_quantized_b200 import sage, sparse
    B, N, H, d, keep = 2, 5000, 24, 64, 7              # more items than two per SM: the counter is in use
    qkv, w, cos, sin = projections(B, N, H, d, 5, cuda_dev)
    nT = -(-N // 128)
    q, k = (torch.empty((B, H, N, d), dtype=torch.bfloat16, device=cuda_dev) for _ in range(2))
    v = torch.empty_like(q)
    lists = torch.empty((B, H, nT, keep), dtype=torch.int32, device=cuda_dev)
    counts = torch.empty((B, H, nT), dtype=torch.int32, device=cuda_dev)
    scratch = sparse.alloc_select_scratch(B, H, N, d, cuda_dev)
    ws = sage.alloc_workspace(B, H, N, d, mode, cuda_dev)
    outs = [torch.empty_like(q) for _ in range(2)]

    def run(o):
        sparse.qk_norm_rope(qkv[:, :, 0], qkv[:, :, 1], wq=w[0], wk=w[1], scope=sparse.NORM_SCOPE_ALL, cos=cos, sin=sin,
                            q_out=q, k_out=k)
        v.copy_(qkv[:, :, 2].permute(0, 2, 1, 3))
        sparse.select_blocks(q, k, keep, lists=lists, counts=counts, scratch=scratch)
        sparse.attn_fwd_sparse(q, k, v, mode, lists, counts, o=o, workspace=ws)

    run(outs[0])
    torch.cuda.synchronize()
    graphs = []
    for o in outs:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            run(o)
        graphs.append(gr)
    for seed in (6, 7):
        fresh, *_ = projections(B, N, H, d, seed, cuda_dev)
        qkv.copy_(fresh)
        ref = layer_ref = torch.empty_like(q)
        run(ref)
        ref = ref.clone()
        for o in outs:
            o.zero_()
        for gr in graphs + graphs:
            gr.replay()
        run(layer_ref)
        torch.cuda.synchronize()
        assert sage.status(ws) == sage.OK
        for o in outs:
            assert torch.equal(bits(o), bits(ref)), seed
        assert torch.equal(bits(layer_ref), bits(ref))


def test_calls_on_other_streams_and_at_once(cuda_dev):
    """The whole run on a given stream while the default stream is busy, and two runs at once on two streams (their
    own workspaces): the bits of the run alone."""
    data = [projections(1, 3000, 8, 128, s, cuda_dev) for s in (11, 12)]
    refs = [layer(*dd, I8, 5)[-1].clone() for dd in data]
    torch.cuda.synchronize()
    busy = torch.randn((4096, 4096), device=cuda_dev)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for rep in range(3):
        for _ in range(4):
            busy = busy @ busy * 1e-3
        outs = []
        for dd, st in zip(data, streams):
            st.wait_stream(torch.cuda.default_stream())
            with torch.cuda.stream(st):                    # v's layout copy runs there, too
                outs.append(layer(*dd, I8, 5, stream=st)[-1])
        for st in streams:
            st.synchronize()
        for o, r in zip(outs, refs):
            assert torch.equal(bits(o), bits(r)), rep


def test_tensors_on_different_devices_are_refused(cuda_dev):
    from video_dit_quantized_b200 import sparse
    q = torch.zeros((1, 2, 200, 64), dtype=torch.bfloat16, device=cuda_dev)
    with pytest.raises(ValueError, match="not a CUDA tensor"):
        sparse.select_blocks(q, q.cpu(), 1)
    with pytest.raises(ValueError, match="not a CUDA tensor"):
        sparse.attn_fwd_sparse(q, q, q, BF16, torch.zeros((1, 2, 2, 1), dtype=torch.int32),
                               torch.zeros((1, 2, 2), dtype=torch.int32))


@pytest.mark.parametrize("B,N,H,d", [(1, 1, 1, 128), (2, 127, 3, 64), (1, 129, 2, 128), (1, 1000, 5, 64), (1, 2000, 3, 128)])
def test_debug_build_is_clean_and_gives_the_same_bits(B, N, H, d, cuda_dev):
    from video_dit_quantized_b200 import sage

    @contextlib.contextmanager
    def debug():
        old = sage.LIB
        sage.LIB = sage.debug_library()
        try:
            yield
        finally:
            sage.LIB = old

    data = projections(B, N, H, d, 20 + N, cuda_dev)
    for mode in (BF16, I8, QTOK):
        ref = layer(*data, mode, 4)
        with debug():
            got = layer(*data, mode, 4)                 # raises on EBOUNDS
        for a, b in zip(got, ref):
            assert torch.equal(bits(a), bits(b))


def test_unaligned_output_rows(cuda_dev):
    """o on a 16-byte boundary only: the narrow stores."""
    from video_dit_quantized_b200 import sparse
    for d in (64, 128):
        q, k, v = (torch.randn((1, 2, 500, d), device=cuda_dev).to(torch.bfloat16) for _ in range(3))
        lists, counts = sparse.select_blocks(q, k, 2)
        pad = torch.zeros(q.numel() + 64, dtype=torch.bfloat16, device=cuda_dev)
        o = pad[8:8 + q.numel()].view(q.shape)
        assert o.data_ptr() % 32 == 16
        for mode in (BF16, I8):
            ref = sparse.attn_fwd_sparse(q, k, v, mode, lists, counts)
            sparse.attn_fwd_sparse(q, k, v, mode, lists, counts, o=o)
            assert torch.equal(bits(o), bits(ref))
            assert (pad[:8] == 0).all() and (pad[8 + q.numel():] == 0).all()


def test_full_lists_have_no_error_against_the_dense_layer(cuda_dev):
    """The library's own error measure between the sparse and the dense output: 0 with all blocks, falling as more
    blocks are kept."""
    from video_dit_quantized_b200 import sage, sparse
    qkv, w, cos, sin = projections(1, 4000, 4, 128, 31, cuda_dev)
    q, k, v, _, _, _ = layer(qkv, w, cos, sin, BF16, 4)
    dense = sage.attn_fwd(q, k, v, BF16)
    errs = []
    for keep in (2, 8, 16, 24, 32):
        lists, counts = sparse.select_blocks(q, k, keep)
        o = sparse.attn_fwd_sparse(q, k, v, BF16, lists, counts)
        errs.append(float(sage.rel_l2(o, dense)))
    assert errs[-1] == 0.0
    assert all(a > b for a, b in zip(errs, errs[1:])), errs


@pytest.mark.parametrize("P,mode", [(1, I8), (2, I8), (4, BF16)])
def test_ulysses_send_of_normed_queries_and_keys(P, mode, cuda_dev):
    """send_qk over P emulated ranks (each with its tokens' tables) is norm, rotation and attention of the whole
    sequence, bit for bit."""
    from video_dit_quantized_b200 import sage, sparse
    from video_dit_quantized_b200.ulysses import UlyssesAttention
    B, N, H, d = 2, 640, 8, 128
    Nl = N // P
    qkv, w, cos, sin = projections(B, N, H, d, 41, cuda_dev)
    norm = dict(wq=w[0], wk=w[1], norm=sparse.NORM_RMS, scope=sparse.NORM_SCOPE_ALL)
    q, k = sparse.qk_norm_rope(qkv[:, :, 0], qkv[:, :, 1], cos=cos, sin=sin, **norm)
    v = qkv[:, :, 2].permute(0, 2, 1, 3).contiguous()
    ref = sage.attn_fwd(q, k, v, mode).permute(0, 2, 1, 3)
    sent = [[] for _ in range(P)]
    ranks = [UlyssesAttention(B, Nl, H, d, P, mode=mode, device=cuda_dev,
                              a2a=lambda out, inp, r=r: sent[r].append((out, inp))) for r in range(P)]

    def exchange():
        for slot in range(len(sent[0])):
            for r in range(P):
                for src in range(P):
                    sent[r][slot][0][src].copy_(sent[src][slot][1][r])
        for s in sent:
            s.clear()

    for again in range(2):
        for r, ua in enumerate(ranks):
            part = qkv[:, r * Nl:(r + 1) * Nl].contiguous()
            ua.send_qk(part[:, :, 0], part[:, :, 1], cos=cos[r * Nl:(r + 1) * Nl], sin=sin[r * Nl:(r + 1) * Nl], **norm)
            ua.send("v", part[:, :, 2])
        exchange()
        for ua in ranks:
            ua.attend_local()
        exchange()
        got = torch.cat([ua.finish().clone() for ua in ranks], dim=1)
        assert torch.equal(bits(got), bits(ref.contiguous())), again
