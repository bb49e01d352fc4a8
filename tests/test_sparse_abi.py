"""include/sage_sparse.h: symbols, binding signatures and refusals, all on the host (no GPU needed)."""
import ctypes
import re

import pytest
import torch

from video_dit_quantized_b200 import sage, sparse

EXPECTED = {"sage_qk_norm_rope", "sage_select_scratch_bytes", "sage_select_blocks", "sage_attn_fwd_sparse",
            "sage_dbg_sparse_forced_timeout"}
VP = ctypes.c_void_p


def test_header_and_libraries_agree():
    assert set(sparse.header_functions()) == EXPECTED
    for lib in (sage.LIB, sage.debug_library()):
        for name in EXPECTED:
            assert hasattr(lib, name), name


def test_binding_signatures_match_the_header():
    txt = re.sub(r"/\*.*?\*/", "", open(sparse.HEADER).read(), flags=re.S)
    kinds = {"int": ctypes.c_int, "size_t": ctypes.c_size_t, "long long": ctypes.c_longlong, "double": ctypes.c_double}
    seen = set()
    for m in re.finditer(r"^(int|size_t)\s+(sage_\w+)\(([^)]*)\);", txt, flags=re.M):
        ret, name, params = m.groups()
        want = [VP if "*" in p else kinds[" ".join(p.split()[:-1])] for p in params.split(",")]
        f = getattr(sage.LIB, name)
        assert list(f.argtypes) == want and f.restype == kinds[ret], name
        seen.add(name)
    assert seen == EXPECTED


def test_header_constants_match_the_binding():
    txt = open(sparse.HEADER).read()
    value = lambda n: int(re.search(rf"#define SAGE_{n} (\d+)", txt).group(1))
    for name in ("NORM_NONE", "NORM_RMS", "NORM_LAYER", "NORM_SCOPE_HEAD", "NORM_SCOPE_ALL", "ROPE_NONE",
                 "ROPE_INTERLEAVED", "ROPE_HALF", "COEFF_DIVIDE", "COEFF_RECIPROCAL", "NORM_MAX_WIDTH", "SELECT_MAX_BLOCKS"):
        assert value(name) == getattr(sparse, name), name


def _norm_args(**kw):
    a = dict(q=1 << 30, k=2 << 30, qs=512, ks=512, wq=3 << 30, bq=None, wk=3 << 30, bk=None, wd=0, cos=4 << 30,
             sin=5 << 30, B=2, N=100, H=4, d=128, norm=sparse.NORM_RMS, scope=0, eps=1e-6, rope=1, begin=0, len=100,
             qo=6 << 30, ko=7 << 30, ranks=0)
    a.update(kw)
    return list(a.values()) + [None]


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), sage.EINVAL), (dict(N=0), sage.EINVAL), (dict(H=0), sage.EINVAL), (dict(d=96), sage.EUNSUPPORTED),
    (dict(H=129, qs=129 * 128, ks=129 * 128), sage.EUNSUPPORTED), (dict(B=1 << 20, N=1 << 12), sage.EINVAL),
    (dict(norm=3), sage.EINVAL), (dict(norm=-1), sage.EINVAL), (dict(scope=2), sage.EINVAL), (dict(rope=3), sage.EINVAL),
    (dict(wd=2), sage.EINVAL), (dict(eps=-1.0), sage.EINVAL), (dict(eps=float("nan")), sage.EINVAL),
    (dict(eps=1e300), sage.EINVAL), (dict(begin=-1), sage.EINVAL), (dict(begin=1), sage.EINVAL),
    (dict(begin=2 ** 31 - 1, len=2 ** 31 - 1), sage.EINVAL), (dict(len=-1), sage.EINVAL), (dict(cos=None), sage.EINVAL),
    (dict(sin=(5 << 30) + 8), sage.EINVAL), (dict(ranks=3), sage.EINVAL), (dict(ranks=-1), sage.EINVAL),
    (dict(q=None), sage.EINVAL),                                     # its output and weight remain
    (dict(q=None, qo=None, wq=None, k=None, ko=None, wk=None), sage.EINVAL),
    (dict(qs=504), sage.EINVAL), (dict(qs=516), sage.EINVAL), (dict(qs=1 << 60), sage.EINVAL),
    (dict(q=(1 << 30) + 8), sage.EINVAL), (dict(qo=(6 << 30) + 8), sage.EINVAL), (dict(wq=(3 << 30) + 8), sage.EINVAL),
    (dict(bq=3 << 30), sage.EINVAL),                                 # RMS has no bias
    (dict(norm=0), sage.EINVAL),                                     # no norm has no weight
    (dict(qo=1 << 30), sage.EINVAL),                                 # onto the input, another layout
    (dict(qo=1 << 30, ranks=1, qs=1024), sage.EINVAL),               # onto a strided input
    (dict(qo=(1 << 30) + 1024, ranks=1), sage.EINVAL),               # shifted onto the input
    (dict(qo=2 << 30, ranks=1), sage.EINVAL),                        # onto the other input
    (dict(ko=6 << 30), sage.EINVAL), (dict(ko=4 << 30), sage.EINVAL), (dict(ko=3 << 30), sage.EINVAL),
])
def test_norm_rope_refusals(kw, code):
    assert sage.LIB.sage_qk_norm_rope(*_norm_args(**kw)) == code


def test_norm_rope_in_place_and_well_formed_calls_reach_the_device_check():
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")
    for kw in (dict(), dict(qo=1 << 30, ko=2 << 30, ranks=1), dict(q=None, qo=None, wq=None), dict(len=0, cos=None, sin=None),
               dict(rope=0, cos=None, sin=None), dict(ranks=4), dict(norm=2, bq=8 << 30)):
        assert sage.LIB.sage_qk_norm_rope(*_norm_args(**kw)) in (sage.ELAUNCH, sage.EUNSUPPORTED), kw


def test_select_refusals():
    f = sage.LIB.sage_select_blocks
    at, odd = [VP((i + 1) << 30) for i in range(5)], VP((1 << 30) + 8)
    n = sparse.select_scratch_bytes(1, 2, 1000, 128)
    rows = 2 * 2 * 8                     # means, three slices, a step and a norm for every block of q and k
    assert n == rows * 128 * 4 + rows * 3 * 128 + 2 * 256
    ok = lambda q=at[0], k=at[1], B=1, H=2, N=1000, d=128, keep=3, first=0, window=0, li=at[2], co=at[3], sc=at[4], nb=n: f(
        q, k, B, H, N, d, keep, first, window, li, co, sc, nb, None)
    for kw in (dict(q=None), dict(k=odd), dict(B=0), dict(N=0), dict(keep=0), dict(first=-1), dict(window=-2),
               dict(window=2), dict(first=3), dict(first=2 ** 31 - 1, window=2 ** 31 - 1), dict(li=None), dict(co=VP(6)),
               dict(sc=odd), dict(H=70000), dict(li=at[0]), dict(co=at[1]), dict(sc=at[0]), dict(sc=at[1]),
               dict(co=at[2]), dict(sc=at[2]), dict(sc=at[3]), dict(li=VP((2 << 30) + 511996))):
        assert ok(**kw) == sage.EINVAL, kw
    assert ok(d=96) == sage.EUNSUPPORTED
    assert ok(nb=n - 1) == sage.EWORKSPACE
    most = sparse.SELECT_MAX_BLOCKS * 128
    assert ok(N=most + 1) == sage.EUNSUPPORTED
    assert sparse.select_scratch_bytes(1, 1, most, 64) > 0 and sparse.select_scratch_bytes(1, 1, most + 1, 64) == 0
    with pytest.raises(sage.SageError):
        sparse.alloc_select_scratch(1, 1, most + 1, 64)
    if not torch.cuda.is_available():
        for kw in (dict(), dict(k=at[0]), dict(li=VP((2 << 30) + 512000))):           # one tensor as q and k; behind k
            assert ok(**kw) in (sage.ELAUNCH, sage.EUNSUPPORTED), kw
        assert ok(keep=8, first=9, window=9) in (sage.ELAUNCH, sage.EUNSUPPORTED)     # every block is kept


def test_sparse_refusals():
    n = sage.workspace_bytes(1, 2, 1000, 128, sage.MODE_INT8_FP8)
    base = dict(q=1 << 30, k=2 << 30, v=3 << 30, o=4 << 30, B=1, H=2, N=1000, d=128, mode=1, li=5 << 30, co=6 << 30,
                width=3, coeff=0, ws=7 << 30, nb=n)
    call = lambda **kw: sage.LIB.sage_attn_fwd_sparse(*{**base, **kw}.values(), None)
    for kw in (dict(q=None), dict(v=(3 << 30) + 8), dict(N=0), dict(mode=3), dict(mode=-1), dict(width=0), dict(coeff=2), dict(coeff=-1), dict(li=None),
               dict(co=(6 << 30) + 2), dict(ws=(7 << 30) + 16), dict(o=1 << 30), dict(o=(2 << 30) + 1024),
               dict(o=5 << 30), dict(o=6 << 30), dict(o=7 << 30), dict(H=70000), dict(ws=1 << 30), dict(ws=2 << 30),
               dict(ws=3 << 30), dict(li=(7 << 30) + 4), dict(co=(7 << 30) + n - 4)):
        assert call(**kw) == sage.EINVAL, kw
    assert call(d=32) == sage.EUNSUPPORTED
    assert call(nb=n - 1) == sage.EWORKSPACE
    dbg = lambda cycles: sage.LIB.sage_dbg_sparse_forced_timeout(*base.values(), cycles, None)
    assert dbg(10) == sage.EINVAL and dbg(1 << 60) == sage.EINVAL
    if not torch.cuda.is_available():
        for kw in (dict(), dict(k=1 << 30, v=1 << 30), dict(co=(7 << 30) + n)):
            assert call(**kw) in (sage.ELAUNCH, sage.EUNSUPPORTED), kw


def test_binding_refuses_what_the_c_abi_cannot_see():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    q = bf(1, 200, 2, 64)
    t = torch.zeros(200, 32)
    for match, args, kw in (
            ("required", (None,), {}), (r"\[B, N, H, d\]", (q[0],), {}), ("bfloat16", (q.float(),), {}),
            ("must not be empty", (q[:, :0],), {}),
            ("shape", (q, bf(1, 100, 2, 64)), {}), ("contiguous", (q.transpose(1, 2),), {}),
            ("contiguous", (q[:, :, :, :32],), {}), ("evenly", (bf(2, 300, 2, 64)[:, :200],), {}),
            ("float32", (q,), dict(cos=t.double(), sin=t.double())), ("shape", (q,), dict(cos=t, sin=t[:, :16].contiguous())),
            ("required", (q,), dict(cos=t)), ("shape", (q,), dict(wq=bf(128))), ("all", (q, q), dict(wq=bf(64), wk=torch.zeros(64))),
            ("all", (q,), dict(wq=torch.zeros(64, dtype=torch.float16))), ("no input", (q,), dict(k_out=bf(1, 2, 200, 64))),
            ("shape", (q,), dict(q_out=bf(1, 200, 2, 64))), ("multiple", (q,), dict(ranks=3)),
            ("not a CUDA tensor", (q, q), dict(wq=bf(64), wk=bf(64), cos=t, sin=t))):
        with pytest.raises(ValueError, match=match):
            sparse.qk_norm_rope(*args, **kw)
    q = bf(1, 2, 200, 64)
    li, co = torch.zeros(1, 2, 2, 1, dtype=torch.int32), torch.zeros(1, 2, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="keep"):
        sparse.select_blocks(q, q, 0)
    with pytest.raises(ValueError, match="shape"):
        sparse.select_blocks(q, q, 2, lists=li)
    with pytest.raises(ValueError, match="bfloat16"):
        sparse.select_blocks(q, q.float(), 1)
    with pytest.raises(ValueError, match="not a CUDA tensor"):
        sparse.select_blocks(q, q, 1)
    with pytest.raises(ValueError, match="shape"):
        sparse.attn_fwd_sparse(q, q, q, 0, li[:, :1].contiguous(), co)
    with pytest.raises(ValueError, match="int32"):
        sparse.attn_fwd_sparse(q, q, q, 0, li.long(), co)
    with pytest.raises(ValueError, match="shape"):
        sparse.attn_fwd_sparse(q, q, q, 0, li, co[:, :1].contiguous())
    with pytest.raises(ValueError, match="not a CUDA tensor"):
        sparse.attn_fwd_sparse(q, q, q, 0, li, co)


def test_ulysses_send_qk_on_the_host():
    """send_qk fills the send layout through norm_rope, starts both exchanges and refuses other shapes (CPU, with a
    stand-in for the kernel: the layout of the send copy)."""
    import sys
    sys.path.insert(0, "tests")
    from _util import attention_seqpar_ref, ulysses_ref_permute
    from video_dit_quantized_b200.ulysses import UlyssesAttention
    calls, sent = [], []

    def norm_rope(q, k, ranks, q_out, k_out, **kw):
        calls.append(kw)
        for x, y in ((q, q_out), (k, k_out)):
            ulysses_ref_permute(2 * x, y, 1, 8, 4, 16, ranks, 0)

    for P in (1, 2):
        calls.clear()
        sent.clear()
        ua = UlyssesAttention(1, 8, 4, 16, P, mode=sage.MODE_BF16, device="cpu", permute=ulysses_ref_permute,
                              attention=attention_seqpar_ref, a2a=lambda o, i: sent.append((o, i)), norm_rope=norm_rope)
        x = torch.randn(1, 8, 4, 16).to(torch.bfloat16)
        with pytest.raises(ValueError, match="k must be"):
            ua.send_qk(x, x[:, :4], eps=1e-5)
        ua.send_qk(x, 3 * x, eps=1e-5)
        assert calls == [dict(eps=1e-5)]
        want = torch.empty(P, 1, 8, 4 // P, 16, dtype=torch.bfloat16)
        ulysses_ref_permute(2 * x, want, 1, 8, 4, 16, P, 0)
        if P == 1:
            assert sent == [] and torch.equal(ua._keep["q"], want)
        else:
            assert [o is ua.recv_buf[t] for (o, _), t in zip(sent, "qk")] == [True, True]
            assert torch.equal(sent[0][1], want)
        with pytest.raises(RuntimeError, match="v"):
            ua.attend_local()


def test_products_of_other_widths_have_columns_of_their_own():
    """Block scores: tcgen05 products run in issue order only where accumulator and shape are the same, so the three
    products (48, 32 and 16 query columns) must not share tensor-memory columns."""
    import os
    from video_dit_quantized_b200 import build
    txt = open(os.path.join(build.CSRC, "select.cu")).read()
    rows = int(re.search(r"constexpr int kRows = (\d+);", txt).group(1))
    cols = int(re.search(r"constexpr uint32_t kAccCols = (\d+);", txt).group(1))
    expr = re.search(r"constexpr int acc_col\(int sl, int qs\) \{ return (.*?); \}", txt).group(1).replace("/", "//")
    at = lambda sl, qs: eval(expr, dict(sl=sl, qs=qs, kRows=rows))
    spans = [range(at(sl, 0), at(sl, 0) + rows * (3 - sl)) for sl in range(3)]
    used = [c for s in spans for c in s]
    assert len(set(used)) == len(used) == 6 * rows and max(used) < cols
    assert [at(sl, qs) for sl in range(3) for qs in range(3 - sl)] == [s[qs * rows] for sl, s in enumerate(spans) for qs in range(3 - sl)]
    assert "mma_ss<kKindI8>(tmem + acc_col(sl, 0)," in txt and "score_idesc(3 - sl), k > 0 ? 1u : 0u)" in txt


def test_reads_ahead_in_a_list_end_with_it():
    """Block-sparse attention reads a list two places ahead.  Widths go up to 2^31 - 1, so the place must be compared
    without adding to the step in 32 bits (which wraps to a negative place, in front of the list)."""
    import os
    import numpy as np
    from video_dit_quantized_b200 import build
    txt = open(os.path.join(build.CSRC, "sparse.cu")).read()
    assert len(re.findall(r"auto listed = \[&\]\(int j, int next\)", txt)) == 2
    assert not re.search(r"listed\(j \+", txt)
    bounds = re.findall(r"return (c|it\.steps) - j > next && SAGE_DCHECK", txt)
    assert sorted(bounds) == ["c", "it.steps"]
    for c in (1, 2, 3, 2 ** 31 - 1):
        for j in {0, max(0, c - 3), max(0, c - 2), c - 1}:
            for ahead in (0, 1, 2):
                assert (np.int64(np.int32(c) - np.int32(j)) > ahead) == (j + ahead < c)
    with np.errstate(over="ignore"):
        assert np.int32(2 ** 31 - 2) + np.int32(2) < 0                        # what the sum would have been


@pytest.mark.parametrize("P", [1, 2])
def test_ulysses_send_qk_refuses_what_it_sets_itself(P):
    """On a stream of its own the norm would still be writing the send buffer when the exchange (or, with one rank,
    attention) reads it: send_qk takes no stream, and no outputs or ranks, and starts nothing."""
    from video_dit_quantized_b200.ulysses import UlyssesAttention
    calls, sent = [], []
    ua = UlyssesAttention(1, 8, 4, 16, P, mode=sage.MODE_BF16, device="cpu", permute=lambda *a: None,
                          attention=lambda *a: None, a2a=lambda o, i: sent.append((o, i)),
                          norm_rope=lambda q, k, **kw: calls.append(kw))
    x = torch.zeros(1, 8, 4, 16, dtype=torch.bfloat16)
    for name, value in (("stream", object()), ("q_out", x), ("k_out", x), ("ranks", 2)):
        with pytest.raises(ValueError, match=name):
            ua.send_qk(x, x, **{name: value})
    assert calls == [] and sent == [] and ua._pending == {} and ua._keep == {}
    ua.send_qk(x, x, eps=1e-5, stream=None)
    assert len(calls) == 1 and "stream" not in calls[0] and calls[0]["eps"] == 1e-5 and len(sent) == (0 if P == 1 else 2)
