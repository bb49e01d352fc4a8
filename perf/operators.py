"""The operators between a DiT's projections and its attention output, as measured work.

Three operators: the per-head (or whole-width) norm of queries and keys with the position rotation in the same
pass, the choice of key blocks from pooled queries and keys, and attention over the chosen blocks in BF16 and
INT8/FP8.  `run` computes them in plain torch operations (own = False) or through the library (own = True);
`exact` computes them from their definitions in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

BLK = 128
NORMS = ("none", "rms", "layer")
ROPES = ("none", "interleaved", "half")
MODES = ("bf16", "int8_fp8", "int8_fp8_qtoken")


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one token: the smallest call, where latency counts (a streamed token, width 5120)
        dict(name="norm_rope_one_token", op="norm_rope", B=1, N=1, H=40, d=128, norm="rms", scope="all", affine=True,
             rope="interleaved", begin=0, rot=1, fused=True, ranks=0),
        # 13x30x45 video tokens behind 226 text tokens that are not rotated, two batch elements, head dim 64,
        # LayerNorm per head with weight and bias
        dict(name="norm_rope_text_video_d64", op="norm_rope", B=2, N=17776, H=30, d=64, norm="layer", scope="head",
             affine=True, rope="interleaved", begin=226, rot=17550, fused=False, ranks=0),
        # one of four sequence-parallel ranks of the 480p model: a quarter of 21x30x52 tokens, written straight
        # into the exchange layout
        dict(name="norm_rope_ranks4", op="norm_rope", B=1, N=8190, H=12, d=128, norm="rms", scope="all", affine=True,
             rope="interleaved", begin=0, rot=8190, fused=True, ranks=4),
        # 21x45x80 tokens of 40 heads out of a fused qkv projection: the 720p model
        dict(name="norm_rope_720p", op="norm_rope", B=1, N=75600, H=40, d=128, norm="rms", scope="all", affine=True,
             rope="interleaved", begin=0, rot=75600, fused=True, ranks=0),
        # a short clip: eight blocks a head
        dict(name="select_short", op="select", B=1, H=2, N=1024, d=128, keep=3, first=0, window=0),
        # text blocks always kept, 20% of the blocks, head dim 64
        dict(name="select_text_video_d64", op="select", B=1, H=30, N=17776, d=64, keep=28, first=2, window=0),
        # a tenth of the blocks of the 720p sequence, neighbours always kept
        dict(name="select_720p", op="select", B=1, H=40, N=75600, d=128, keep=59, first=0, window=1),
        # a short, odd clip in BF16
        dict(name="sparse_bf16_short", op="sparse", B=1, H=2, N=1000, d=128, mode="bf16", keep=3, lists="even"),
        # 20% density at head dim 64 in BF16
        dict(name="sparse_bf16_d64", op="sparse", B=1, H=30, N=17776, d=64, mode="bf16", keep=28, lists="even"),
        # lists of every length from 0 to 64, in no order: a learned or cached pattern on the 480p sequence
        dict(name="sparse_bf16_ragged", op="sparse", B=1, H=12, N=32760, d=128, mode="bf16", keep=64, lists="ragged"),
        # per-token query scales, ragged lists, two batch elements, head dim 64
        dict(name="sparse_qtoken_ragged", op="sparse", B=2, H=30, N=17776, d=64, mode="int8_fp8_qtoken", keep=28,
             lists="ragged"),
        # a tenth of the 720p sequence in INT8/FP8, the largest call
        dict(name="sparse_i8f8_720p", op="sparse", B=1, H=40, N=75600, d=128, mode="int8_fp8", keep=59, lists="even"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm_rope", "select", "sparse", "sparse"))
    least = rng.choice((1, 64, 512, 512))
    d = rng.choice((64, 128))
    B = rng.choice((1, 1, 2, 3))
    H = rng.choice((1, 2, 3, 5, 8, 12, 16, 24, 30, 40))
    if op == "norm_rope":
        cap = 75600 * 40 * 128 // (B * H * d)
        N = _log_int(rng, least, min(75600, cap))
        begin = rng.choice((0, 0, min(N, 226), rng.randint(0, N)))
        rot = rng.choice((N - begin, rng.randint(0, N - begin)))
        rope = rng.choice(ROPES)
        divisors = [p for p in (2, 3, 4, 5, 8) if H % p == 0]
        return dict(op=op, B=B, N=N, H=H, d=d, norm=rng.choice(NORMS[1:] if rope == "none" else NORMS), scope=rng.choice(("head", "all")),
                    affine=rng.random() < 0.8, rope=rope, begin=begin, rot=rot,
                    fused=rng.random() < 0.5, ranks=rng.choice([0, 0, 1] + divisors))
    if op == "select":
        cap = 75600 * 40 * 128 // (B * H * d)
        N = _log_int(rng, least, min(75600, cap))
        nT = -(-N // BLK)
        keep = rng.randint(1, max(1, nT // 3)) if rng.random() < 0.8 else nT + 2
        window = rng.choice((-1, 0, 0, 1, 2))
        first = rng.choice((0, 0, 1, 2))
        while max(0, 2 * window + 1) + first > keep:
            window, first = (window - 1, first) if window >= 0 else (window, first - 1)
        return dict(op=op, B=B, H=H, N=N, d=d, keep=keep, first=first, window=window)
    cap = 75600 * 40 * 128 // (B * H * d)
    N = _log_int(rng, least, min(75600, cap))
    nT = -(-N // BLK)
    most = max(1, int(0.5 * 40 * 591 * 59 * 128 // (B * H * nT * d)))       # half the largest case's products
    keep = rng.randint(1, max(1, min(nT, most)))
    return dict(op=op, B=B, H=H, N=N, d=d, mode=rng.choice(MODES), keep=keep, lists=rng.choice(("even", "ragged")))


# ------------------------------------------------------------------------------------------------ inputs

def _angles(rot, d):
    """fp64 angles [rot, d/2] of a (frame, row, column) position grid, the channel pairs split in three."""
    w = 80 if rot > 40000 else 52 if rot > 2000 else 8
    h = 45 if rot > 40000 else 30 if rot > 2000 else 4
    n = torch.arange(rot, device="cuda", dtype=torch.float64)
    pos = (torch.div(n, h * w, rounding_mode="floor"), torch.div(n, w, rounding_mode="floor") % h, n % w)
    half = d // 2
    third = half // 3
    parts = []
    for p, m in zip(pos, (half - 2 * third, third, third)):
        freq = 10000.0 ** (-torch.arange(m, device="cuda", dtype=torch.float64) / m)
        parts.append(p[:, None] * freq[None, :])
    return torch.cat(parts, dim=1)


def _video_qkv(g, B, H, N, d, parts):
    """bf16 [B,H,N,d]: a slowly varying part shared by neighbouring tokens, noise, K with channel offsets."""
    nT = -(-N // BLK)
    out = []
    for p in parts:
        x = torch.randn((B, H, N, d), generator=g, device="cuda", dtype=torch.float32)
        if p != "v":
            slow = torch.randn((B, H, nT, d), generator=g, device="cuda") * 0.5
            x += slow.repeat_interleave(BLK, dim=2)[:, :, :N]
        if p == "k":
            x += 3.0 * torch.randn((B, H, 1, d), generator=g, device="cuda")
        out.append(x.to(torch.bfloat16))
        del x
    return out


def _block_lists(g, B, H, nT, keep, kind):
    """int32 lists [B,H,nT,keep] and counts [B,H,nT]: distinct blocks, -1 behind the count."""
    G = B * H * nT
    score = torch.rand((G, nT), generator=g, device="cuda")
    own_block = torch.arange(nT, device="cuda").repeat(B * H)
    score[torch.arange(G, device="cuda"), own_block] = 2.0
    order = score.argsort(dim=1, descending=True)[:, :keep]
    if kind == "even":
        lists = order.sort(dim=1).values
        counts = torch.full((G,), keep, device="cuda", dtype=torch.int64)
    else:
        lists = order
        counts = torch.randint(0, keep + 1, (G,), generator=g, device="cuda")
    lists = lists.masked_fill(torch.arange(keep, device="cuda")[None, :] >= counts[:, None], -1)
    return (lists.to(torch.int32).view(B, H, nT, keep).contiguous(),
            counts.to(torch.int32).view(B, H, nT).contiguous())


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, B, N, H, d = case["op"], case["B"], case["N"], case["H"], case["d"]
    st = dict(case=case)
    if op == "norm_rope":
        if case["fused"]:                      # slices of one projection's output
            qkv = torch.randn((B, N, 3, H, d), generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)
            st["q"], st["k"] = qkv[:, :, 0], qkv[:, :, 1]
        else:
            st["q"], st["k"] = (torch.randn((B, N, H, d), generator=g, device="cuda").to(torch.bfloat16)
                                for _ in range(2))
        width = d if case["scope"] == "head" else H * d
        affine = case["affine"] and case["norm"] != "none"
        for name in ("wq", "wk"):
            st[name] = ((1.0 + 0.2 * torch.randn(width, generator=g, device="cuda")).to(torch.bfloat16)
                        if affine else None)
        for name in ("bq", "bk"):
            st[name] = ((0.1 * torch.randn(width, generator=g, device="cuda")).to(torch.bfloat16)
                        if affine and case["norm"] == "layer" else None)
        st["cos"] = st["sin"] = None
        if case["rope"] != "none":
            a = _angles(case["rot"], d)
            st["cos"], st["sin"] = a.cos().float().contiguous(), a.sin().float().contiguous()
        P = case["ranks"]
        shape = (B, H, N, d) if P == 0 else (P, B, N, H // P, d)
        st["q_out"], st["k_out"] = (torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        return st
    nT = -(-N // BLK)
    if op == "select":
        st["q"], st["k"] = _video_qkv(g, B, H, N, d, "qk")
        st["lists"] = torch.empty((B, H, nT, case["keep"]), dtype=torch.int32, device="cuda")
        st["counts"] = torch.empty((B, H, nT), dtype=torch.int32, device="cuda")
        if own:
            from video_dit_quantized_b200 import sparse
            st["scratch"] = sparse.alloc_select_scratch(B, H, N, d, st["q"].device)
        return st
    st["q"], st["k"], st["v"] = _video_qkv(g, B, H, N, d, "qkv")
    st["lists"], st["counts"] = _block_lists(g, B, H, nT, case["keep"], case["lists"])
    st["o"] = torch.empty_like(st["q"])
    if own:
        from video_dit_quantized_b200 import sage
        st["mode"] = MODES.index(case["mode"])
        st["workspace"] = sage.alloc_workspace(B, H, N, d, st["mode"], st["q"].device)
    return st


# ------------------------------------------------------------------------------------------------ one pass

def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        return _run_own(state, case, op)
    if op == "norm_rope":
        return [_norm_rope_plain(state[t], state["w" + t], state["b" + t], state["cos"], state["sin"], case)
                for t in "qk"]
    if op == "select":
        return _select_plain(state["q"], state["k"], case)
    if case["mode"] == "bf16":
        return _sparse_plain(state["q"], state["k"], state["v"], state["lists"], state["counts"])
    return _sparse_quant_plain(state["q"], state["k"], state["v"], state["lists"], state["counts"],
                               case["mode"] == "int8_fp8_qtoken")


def _run_own(state, case, op):
    from video_dit_quantized_b200 import sparse
    if op == "norm_rope":
        q, k = sparse.qk_norm_rope(state["q"], state["k"], wq=state["wq"], wk=state["wk"], bq=state["bq"],
                                   bk=state["bk"], norm=NORMS.index(case["norm"]),
                                   scope=sparse.NORM_SCOPE_HEAD if case["scope"] == "head" else sparse.NORM_SCOPE_ALL,
                                   eps=1e-6, cos=state["cos"], sin=state["sin"], rope=ROPES.index(case["rope"]),
                                   rope_begin=case["begin"], ranks=case["ranks"], q_out=state["q_out"],
                                   k_out=state["k_out"])
        return [q, k]
    if op == "select":
        lists, counts = sparse.select_blocks(state["q"], state["k"], case["keep"], first=case["first"],
                                             window=case["window"], lists=state["lists"], counts=state["counts"],
                                             scratch=state["scratch"])
        return [lists, counts]
    return sparse.attn_fwd_sparse(state["q"], state["k"], state["v"], state["mode"], state["lists"], state["counts"],
                                  coeff=sparse.COEFF_RECIPROCAL, o=state["o"], workspace=state["workspace"])


# ------------------------------------------------------------------------------------------------ plain forms

def _norm_rope_plain(x, w, b, cos, sin, case):
    """x bf16 [B,N,H,d] -> norm, rotation, output layout; fp32, rounded once."""
    B, N, H, d = x.shape
    y = x.float()
    if case["scope"] == "all":
        y = y.reshape(B, N, 1, H * d)
    if case["norm"] == "rms":
        y = y * torch.rsqrt((y * y).mean(dim=-1, keepdim=True) + 1e-6)
    elif case["norm"] == "layer":
        y = y - y.mean(dim=-1, keepdim=True)
        y = y * torch.rsqrt((y * y).mean(dim=-1, keepdim=True) + 1e-6)
    if w is not None:
        y = y * w.float()
    if b is not None:
        y = y + b.float()
    y = y.reshape(B, N, H, d)
    if cos is not None and case["rot"] > 0:
        lo, hi = case["begin"], case["begin"] + case["rot"]
        r = y[:, lo:hi]
        a, c = (r[..., 0::2], r[..., 1::2]) if case["rope"] == "interleaved" else (r[..., :d // 2], r[..., d // 2:])
        co, si = cos[None, :, None, :], sin[None, :, None, :]
        ra, rc = a * co - c * si, a * si + c * co
        r = torch.stack((ra, rc), dim=-1).flatten(-2) if case["rope"] == "interleaved" else torch.cat((ra, rc), dim=-1)
        y = torch.cat((y[:, :lo], r, y[:, hi:]), dim=1)
    P = case["ranks"]
    if P == 0:
        y = y.permute(0, 2, 1, 3)
    else:
        y = y.reshape(B, N, P, H // P, d).permute(2, 0, 1, 3, 4)
    return y.to(torch.bfloat16).contiguous()


def _pooled(x):
    """fp32 [B,H,nT,d]: the mean of every 128-token block, summed in fp64 (scores near a border decide)."""
    B, H, N, d = x.shape
    nT = -(-N // BLK)
    full = N // BLK
    sums = []
    if full:
        sums.append(x[:, :, :full * BLK].reshape(B, H, full, BLK, d).sum(dim=3, dtype=torch.float64))
    if full < nT:
        sums.append(x[:, :, full * BLK:].sum(dim=2, keepdim=True, dtype=torch.float64))
    s = torch.cat(sums, dim=2)
    rows = torch.full((nT,), BLK, dtype=torch.float64, device=x.device)
    rows[-1] = N - (nT - 1) * BLK
    return (s / rows[:, None]).float()


def _select_plain(q, k, case):
    B, H, N, d = q.shape
    nT, keep = -(-N // BLK), case["keep"]
    score = torch.matmul(_pooled(q).double(), _pooled(k).double().transpose(-1, -2))
    i = torch.arange(nT, device=q.device)
    forced = (i[None, :] < case["first"]).expand(nT, nT) | ((i[:, None] - i[None, :]).abs() <= case["window"])
    score = score.masked_fill(forced, float("inf"))
    n = min(keep, nT)
    best = score.sort(dim=-1, descending=True, stable=True).indices[..., :n].sort(dim=-1).values
    lists = torch.full((B, H, nT, keep), -1, dtype=torch.int32, device=q.device)
    lists[..., :n] = best
    counts = torch.full((B, H, nT), n, dtype=torch.int32, device=q.device)
    return [lists, counts]


def _blocks(x, fill=0.0):
    """[BH, N, d] -> fp32 [BH, nT, 128, d], rows past N zero."""
    BH, N, d = x.shape
    nT = -(-N // BLK)
    out = torch.zeros((BH, nT * BLK, d), dtype=torch.float32, device=x.device)
    out[:, :N] = x
    return out.view(BH, nT, BLK, d)


def _sparse_plain(q, k, v, lists, counts):
    """softmax(q k^T / sqrt(d)) v over the listed blocks, a group of query blocks at a time."""
    B, H, N, d = q.shape
    BH, nT, keep = B * H, lists.shape[2], lists.shape[3]
    lists, counts = lists.view(BH, nT, keep).long(), counts.view(BH, nT)
    o = torch.empty((BH, nT * BLK, d), dtype=torch.bfloat16, device=q.device)
    step = max(1, (1 << 29) // (BLK * BLK * keep * 4))
    col = torch.arange(BLK, device=q.device)
    slot = torch.arange(keep, device=q.device)
    q, k, v = q.view(BH, N, d), k.view(BH, N, d), v.view(BH, N, d)
    for h in range(BH):
        qb, kb, vb = (_blocks(x[h:h + 1])[0] for x in (q, k, v))
        for i0 in range(0, nT, step):
            i1 = min(nT, i0 + step)
            j = lists[h, i0:i1].clamp(min=0)                                   # [n, keep]
            live = (slot[None, :] < counts[h, i0:i1, None])[:, :, None] & (j[:, :, None] * BLK + col < N)
            s = torch.bmm(qb[i0:i1], kb[j].view(i1 - i0, keep * BLK, d).transpose(1, 2)) / math.sqrt(d)
            s = s.masked_fill(~live.view(i1 - i0, 1, keep * BLK), float("-inf"))
            m = s.amax(dim=-1, keepdim=True).clamp(min=-3e38)
            p = torch.exp(s - m)
            l = p.sum(dim=-1, keepdim=True)
            r = torch.bmm(p, vb[j].view(i1 - i0, keep * BLK, d))
            o[h, i0 * BLK:i1 * BLK] = torch.where(l > 0, r / l.clamp(min=1e-30), 0.0).view(-1, d).to(torch.bfloat16)
    return o[:, :N].reshape(B, H, N, d)


def _codes(x, dims):
    """INT8 codes (as fp32) and scale of fp32 x with one scale per group over dims; an all-zero group gets 0."""
    amax = x.abs().amax(dim=dims, keepdim=True)
    inv = torch.where(amax > 0, 127.0 / amax, 0.0)
    return (x * inv).round().clamp(-127, 127), amax / 127.0


def _sparse_quant_plain(q, k, v, lists, counts, per_token):
    """The INT8/FP8 scheme over the listed blocks, block by block in list order with a running maximum."""
    B, H, N, d = q.shape
    BH, nT, keep = B * H, lists.shape[2], lists.shape[3]
    q, k, v = q.view(BH, N, d), k.view(BH, N, d), v.view(BH, N, d)
    ks = k.float() - k.double().mean(dim=1, keepdim=True).float()
    qc, qs = _codes(_blocks(q), (-1,) if per_token else (-2, -1))              # scale [BH,nT,128|1,1]
    kc, kscale = _codes(_blocks(ks), (-2, -1))
    del ks
    vmax = v.abs().amax(dim=1, keepdim=True).float()
    v8 = (v.float() * torch.where(vmax > 0, 448.0 / vmax, 0.0)).clamp(-448, 448).to(torch.float8_e4m3fn).float()
    v8, vscale = _blocks(v8), vmax / 448.0
    c = torch.tensor(1.4426950408889634 / math.sqrt(d), dtype=torch.float32, device=q.device)
    lists, counts = lists.view(BH, nT, keep).long(), counts.view(BH, nT)
    o = torch.empty((BH, nT * BLK, d), dtype=torch.bfloat16, device=q.device)
    col = torch.arange(BLK, device=q.device)
    heads = max(1, 4096 // nT)
    for h0 in range(0, BH, heads):
        h1 = min(BH, h0 + heads)
        hs = torch.arange(h0, h1, device=q.device)[:, None].expand(-1, nT).reshape(-1)
        G = (h1 - h0) * nT
        qg, sg = qc[h0:h1].reshape(G, BLK, d), qs[h0:h1].reshape(G, -1, 1)
        m = torch.full((G, BLK, 1), float("-inf"), device=q.device)
        l = torch.zeros((G, BLK, 1), device=q.device)
        acc = torch.zeros((G, BLK, d), device=q.device)
        for t in range(keep):
            j = lists[h0:h1, :, t].reshape(-1).clamp(min=0)
            live = (t < counts[h0:h1].reshape(-1))[:, None] & (j[:, None] * BLK + col < N)
            s = torch.bmm(qg, kc[hs, j].transpose(1, 2)) * ((sg * kscale[hs, j].view(G, 1, 1)) * c)
            s = s.masked_fill(~live[:, None, :], float("-inf"))
            m_new = torch.maximum(m, s.amax(dim=-1, keepdim=True))
            base = m_new.clamp(min=-3e38)
            p = torch.exp2(s - base)
            alpha = torch.exp2(m - base)
            l = l * alpha + p.sum(dim=-1, keepdim=True)
            p8 = (p * 448.0).to(torch.float8_e4m3fn).float()
            acc = acc * alpha + torch.bmm(p8, v8[hs, j])
            m = m_new
        r = torch.where(l > 0, acc * vscale[hs] / (448.0 * l.clamp(min=1e-30)), 0.0)
        o[h0:h1] = r.view(h1 - h0, nT * BLK, d).to(torch.bfloat16)
    return o[:, :N].reshape(B, H, N, d)


# ------------------------------------------------------------------------------------------------ the work

def work(case):
    B, N, H, d = case["B"], case["N"], case["H"], case["d"]
    nT = -(-N // BLK)
    tensor = 2 * B * N * H * d                                                # bytes of one bf16 tensor
    if case["op"] == "norm_rope":
        tables = 2 * 4 * case["rot"] * d // 2 if case["rope"] != "none" else 0
        per = (0, 4, 8)[NORMS.index(case["norm"])] + (0 if case["rope"] == "none" else 3)
        return {"bytes": 4 * tensor + tables, "flops": 2 * B * N * H * d * per}
    if case["op"] == "select":
        return {"bytes": 2 * tensor + 4 * B * H * nT * (case["keep"] + 1),
                "flops": 2 * B * H * nT * nT * d + 2 * B * H * N * d}
    share = 1.0 if case["lists"] == "even" else 0.5
    pairs = B * H * N * min(N, share * case["keep"] * BLK)
    return {"bytes": 4 * tensor + 4 * B * H * nT * (case["keep"] + 1), "flops": int(4 * d * pairs)}


# ------------------------------------------------------------------------------------------------ 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm_rope":
        return [_norm_rope_exact(st, t) for t in "qk"]
    if case["op"] == "select":
        return _select_exact(st["q"], st["k"], case)
    q, k, v = st["q"], st["k"], st["v"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    for b in range(case["B"]):
        for h in range(case["H"]):
            args = (q[b, h], k[b, h], v[b, h], st["lists"][b, h], st["counts"][b, h])
            out[b, h] = (_head_exact(*args) if case["mode"] == "bf16"
                         else _head_quant_exact(*args, case["mode"] == "int8_fp8_qtoken"))
    return out


def _norm_rope_exact(st, t):
    case = st["case"]
    B, N, H, d = case["B"], case["N"], case["H"], case["d"]
    w, b = st["w" + t], st["b" + t]
    P = case["ranks"]
    out = torch.empty(st["q_out"].shape, dtype=torch.float64, device="cuda")
    for h0 in range(0, N, 8192):                                               # a group of tokens at a time
        h1 = min(N, h0 + 8192)
        y = st[t][:, h0:h1].double()
        dims = (2, 3) if case["scope"] == "all" else (3,)
        if case["norm"] == "layer":
            y = y - y.mean(dim=dims, keepdim=True)
        if case["norm"] != "none":
            y = y / torch.sqrt(y.square().mean(dim=dims, keepdim=True) + 1e-6)
        if w is not None:
            y = y * w.double().view((H, d) if case["scope"] == "all" else (1, d))
        if b is not None:
            y = y + b.double().view((H, d) if case["scope"] == "all" else (1, d))
        lo, hi = max(h0, case["begin"]), min(h1, case["begin"] + case["rot"])
        if case["rope"] != "none" and lo < hi:
            co = st["cos"].double()[lo - case["begin"]:hi - case["begin"]]
            si = st["sin"].double()[lo - case["begin"]:hi - case["begin"]]
            z = torch.complex(co, si)[None, :, None, :]
            r = y[:, lo - h0:hi - h0]
            if case["rope"] == "interleaved":
                turned = torch.view_as_real(torch.complex(r[..., 0::2].contiguous(), r[..., 1::2].contiguous()) * z)
                y[:, lo - h0:hi - h0] = turned.reshape(r.shape)
            else:
                turned = torch.complex(r[..., :d // 2].contiguous(), r[..., d // 2:].contiguous()) * z
                y[:, lo - h0:hi - h0] = torch.cat((turned.real, turned.imag), dim=-1)
        for h in range(H):
            if P == 0:
                out[:, h, h0:h1] = y[:, :, h]
            else:
                out[h // (H // P), :, h0:h1, h % (H // P)] = y[:, :, h]
    return out


def _select_exact(q, k, case):
    B, H, N, d = q.shape
    nT, keep = -(-N // BLK), case["keep"]
    lists = torch.full((B, H, nT, keep), -1, dtype=torch.int32, device=q.device)
    counts = torch.full((B, H, nT), min(keep, nT), dtype=torch.int32, device=q.device)
    block = torch.arange(N, device=q.device) // BLK
    rows = torch.bincount(block, minlength=nT).double()
    for b in range(B):
        for h in range(H):
            pooled = []
            for x in (q[b, h], k[b, h]):
                s = torch.zeros((nT, d), dtype=torch.float64, device=q.device)
                s.index_add_(0, block, x.double())
                pooled.append((s / rows[:, None]).float().double())
            for i0 in range(0, nT, 64):
                i1 = min(nT, i0 + 64)
                s = (pooled[0][i0:i1, None, :] * pooled[1][None, :, :]).sum(dim=-1)
                for i in range(i0, i1):
                    s[i - i0, :case["first"]] = float("inf")
                    if case["window"] >= 0:
                        s[i - i0, max(0, i - case["window"]):i + case["window"] + 1] = float("inf")
                rank = torch.argsort(-s, dim=1, stable=True)[:, :keep]
                lists[b, h, i0:i1, :rank.shape[1]] = torch.sort(rank, dim=1).values.to(torch.int32)
    return [lists, counts]


def _pad64(x, nT):
    return torch.cat((x, x.new_zeros((nT * BLK - x.shape[0], x.shape[1])))).view(nT, BLK, -1)


def _head_exact(q, k, v, lists, counts):
    N, d = q.shape
    nT, keep = lists.shape
    qb, kb, vb = (_pad64(x.double(), nT) for x in (q, k, v))
    real = torch.arange(nT * BLK, device=q.device).view(nT, BLK) < N
    out = torch.zeros((nT, BLK, d), dtype=torch.float64, device=q.device)
    step = max(1, (1 << 28) // (BLK * BLK * keep * 8))
    for i0 in range(0, nT, step):
        ll, cc = lists[i0:i0 + step].long(), counts[i0:i0 + step]
        n = ll.shape[0]
        ok = (torch.arange(keep, device=q.device) < cc[:, None])
        ll = torch.where(ok, ll, 0)
        keys = (real[ll] & ok[:, :, None]).reshape(n, 1, keep * BLK)
        s = qb[i0:i0 + n] @ kb[ll].reshape(n, keep * BLK, d).mT * d ** -0.5
        s = torch.where(keys, s, -math.inf)
        some = keys.any(dim=-1)[:, 0]
        p = torch.softmax(s[some], dim=-1)
        r = out[i0:i0 + n]
        r[some] = p @ vb[ll].reshape(n, keep * BLK, d)[some]
    return out.view(nT * BLK, d)[:N]


def _head_quant_exact(q, k, v, lists, counts, per_token):
    """One head of the INT8/FP8 scheme in fp64; only the roundings that define the scheme are made."""
    N, d = q.shape
    nT, keep = lists.shape

    def int8(x, dims):                        # the scheme's fp32 code formula, and its fp32 scale
        amax = x.abs().amax(dim=dims, keepdim=True)
        inv = torch.where(amax > 0, 127.0 / amax, torch.zeros_like(amax))
        return torch.clamp(torch.round(x * inv), -127, 127).double(), (amax / 127.0).double()

    mean = (k.double().sum(dim=0) / N).float()
    qi, qs = int8(_pad64(q.float(), nT), (2,) if per_token else (1, 2))
    ki, ks = int8(_pad64(k.float() - mean, nT), (1, 2))
    vmax = v.float().abs().amax(dim=0)
    inv = torch.where(vmax > 0, 448.0 / vmax, torch.zeros_like(vmax))
    v8 = _pad64(torch.clamp(v.float() * inv, -448, 448).to(torch.float8_e4m3fn).double(), nT)
    vs = (vmax / 448.0).double()
    real = torch.arange(nT * BLK, device=q.device).view(nT, 1, BLK) < N
    top = torch.full((nT, BLK, 1), -math.inf, dtype=torch.float64, device=q.device)
    total = torch.zeros_like(top)
    acc = torch.zeros((nT, BLK, d), dtype=torch.float64, device=q.device)
    for t in range(keep):
        use = (counts > t).nonzero()[:, 0]
        if use.numel() == 0:
            break
        j = lists[use, t].long()
        s = (qi[use] @ ki[j].mT) * (qs[use] * ks[j]) * (math.log2(math.e) / math.sqrt(d))
        s = torch.where(real[j], s, -math.inf)
        high = torch.maximum(top[use], s.amax(dim=-1, keepdim=True))
        p = torch.exp2(s - high)
        down = torch.exp2(top[use] - high)
        p8 = (p * 448.0).float().to(torch.float8_e4m3fn).double()
        acc[use] = acc[use] * down + p8 @ v8[j]
        total[use] = total[use] * down + p.sum(dim=-1, keepdim=True)
        top[use] = high
    out = torch.where(total > 0, acc * vs / (448.0 * total), torch.zeros_like(acc))
    return out.view(nT * BLK, d)[:N]
