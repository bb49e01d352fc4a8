"""Block-sparse attention and the steps before it (include/sage_sparse.h).

    q, k = sparse.qk_norm_rope(q, k, wq=..., wk=..., cos=cos, sin=sin)   # projections -> [B, H, N, d]
    lists, counts = sparse.select_blocks(q, k, keep)                    # key blocks of every query block
    o = sparse.attn_fwd_sparse(q, k, v, mode, lists, counts)            # attention over them

Argument marshalling only, as in sage.py; the kernels are in libsage.so.
Every call runs on the device of its tensors, whichever device is current, on
`stream` or on that device's current stream.  Tensors that a call allocates
itself are kept from reuse until the work on `stream` is done.
"""
from __future__ import annotations

import os
import re

import torch

from . import sage
from .sage import BLK, EINVAL, SageError, _check, _need

NORM_NONE, NORM_RMS, NORM_LAYER = 0, 1, 2
NORM_SCOPE_HEAD, NORM_SCOPE_ALL = 0, 1
ROPE_NONE, ROPE_INTERLEAVED, ROPE_HALF = 0, 1, 2
COEFF_DIVIDE, COEFF_RECIPROCAL = 0, 1
NORM_MAX_WIDTH = 16384
SELECT_MAX_BLOCKS = 6016

HEADER = os.path.join(os.path.dirname(sage.HEADER), "sage_sparse.h")


def _where(stream, names: str, *tensors):
    """Index of the one CUDA device all given tensors (None: left out) and the stream belong to."""
    where = {t.get_device() for t in tensors if t is not None}
    dev = where.pop()
    if dev < 0 or where:
        dev = -1
        for name, t in zip(names.split(), tensors):
            if t is None:
                continue
            d = t.get_device()
            if d < 0:
                raise ValueError(f"{name}: a tensor passed for device memory is not a CUDA tensor")
            dev = d if dev < 0 else dev
            if d != dev:
                raise ValueError(f"{name} is on cuda:{d}, the other tensors on cuda:{dev}")
    if stream is not None and stream.device.index != dev:
        raise ValueError(f"the stream belongs to {stream.device}, the tensors to cuda:{dev}")
    return dev


def _handle(stream, dev: int) -> int:
    """The stream to launch on: the given one, or the device's current one."""
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(dev)


def _launch(what: str, dev: int, *args):
    """Calls a C entry point with the tensors' device current."""
    f = getattr(sage.LIB, what)
    if torch._C._cuda_getDevice() == dev:
        rc = f(*args)
    else:
        with torch.cuda.device(dev):
            rc = f(*args)
    _check(rc, what)


def _new(like, shape, dtype, stream, zeroed: int = 0):
    """Memory on the device of `like` made for one call, of the stream that the call runs on: its first elements
    zeroed there, and not given to anyone else before that stream is done with it."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return _new(like, shape, dtype, None, zeroed)
    t = like.new_empty(shape, dtype=dtype)
    if zeroed:
        t[:zeroed].zero_()
    return t


def _is(t, name, dtype, shape, optional=False):
    """_need, with the checks of a good tensor in one expression."""
    if t is None:
        if not optional:
            _need(t, name, dtype, shape)
    elif t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        _need(t, name, dtype, shape)


def _p(t):
    return None if t is None else t.data_ptr()


def header_functions() -> list[str]:
    """Names of the functions declared in include/sage_sparse.h."""
    txt = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return re.findall(r"^\s*(?:const\s+)?[A-Za-z_][\w\s\*]*?\b([a-z_][a-z0-9_]*)\s*\(", txt, flags=re.M)


def _rows(t, name, shape):
    """Row stride in elements of a [B, N, H, d] tensor whose H * d channels are contiguous and whose batches
    follow one another."""
    if t.dtype is not torch.bfloat16:
        raise ValueError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    B, N, H, d = shape
    sb, sn, sh, sd = t.stride()
    # the stride of a dimension of one element says nothing
    row = sn if N > 1 else (sb if B > 1 else H * d)
    if (sd != 1 and d > 1) or (sh != d and H > 1) or (B > 1 and sb != N * row):
        raise ValueError(f"{name}: the channels of a token must be contiguous and the tokens evenly spaced")
    return row


def qk_norm_rope(q, k=None, wq=None, wk=None, bq=None, bk=None, norm: int = NORM_RMS, scope: int = NORM_SCOPE_HEAD,
                 eps: float = 1e-6, cos=None, sin=None, rope: int = ROPE_INTERLEAVED, rope_begin: int = 0, ranks: int = 0,
                 q_out=None, k_out=None, stream=None):
    """Norm of q and k [B, N, H, d] (slices of a fused projection as they are) and the position rotation, written
    in the layout that attention reads: [B, H, N, d], or with ranks = P >= 1 the exchange layout
    [P, B, N, H/P, d].  Returns (q_out, k_out); q or k may be None.

    cos, sin: fp32 [rope_len, d/2] for the tokens rope_begin .. rope_begin + rope_len - 1 (ignored with
    ROPE_NONE; without tables nothing is rotated).  Weights: bf16 or fp32, all of one type, [d] (per head) or
    [H * d] (over all heads).
    """
    x = q if q is not None else k
    if x is None:
        raise ValueError("q or k is required")
    if x.dim() != 4:
        raise ValueError("q and k must be [B, N, H, d]")
    B, N, H, d = shape = tuple(x.shape)
    if 0 in shape:
        raise ValueError("q and k must not be empty")
    if rope == ROPE_NONE or (cos is None and sin is None):
        rope, cos, sin, rope_len = ROPE_NONE, None, None, 0
        rope_begin = 0
    else:
        if cos is None or cos.dim() != 2:
            _need(cos, "cos", torch.float32, ("rope_len", d // 2))
        rope_len = cos.shape[0]
        _is(cos, "cos", torch.float32, (rope_len, d // 2))
        _is(sin, "sin", torch.float32, (rope_len, d // 2))
    w_dtype = None
    width = (H * d,) if scope == NORM_SCOPE_ALL else (d,)
    for t, name in ((wq, "wq"), (bq, "bq"), (wk, "wk"), (bk, "bk")):
        if t is None:
            continue
        w_dtype = w_dtype or t.dtype
        if t.dtype != w_dtype or t.dtype not in (torch.bfloat16, torch.float32):
            raise ValueError(f"{name}: the weights must all be bfloat16 or all float32")
        _is(t, name, w_dtype, width)
    q_row = 0 if q is None else _rows(q, "q", shape)
    k_row = 0 if k is None else _rows(k, "k", shape)
    if ranks < 0 or (ranks > 0 and H % ranks):
        raise ValueError(f"H={H} must be a multiple of ranks={ranks}")
    out_shape = (ranks, B, N, H // ranks, d) if ranks else (B, H, N, d)
    for src, t, name in ((q, q_out, "q_out"), (k, k_out, "k_out")):
        if src is None and t is not None:
            raise ValueError(f"{name} has no input")
        _is(t, name, torch.bfloat16, out_shape, optional=True)
    dev = _where(stream, "q k wq wk bq bk cos sin q_out k_out", q, k, wq, wk, bq, bk, cos, sin, q_out, k_out)
    if q is not None and q_out is None:
        q_out = _new(q, out_shape, torch.bfloat16, stream)
    if k is not None and k_out is None:
        k_out = _new(k, out_shape, torch.bfloat16, stream)
    _launch("sage_qk_norm_rope", dev, _p(q), _p(k), q_row, k_row, _p(wq), _p(bq), _p(wk), _p(bk),
            sage.DTYPE_F32 if w_dtype == torch.float32 else sage.DTYPE_BF16, _p(cos), _p(sin), B, N, H, d, int(norm),
            int(scope), float(eps), int(rope), int(rope_begin), rope_len, _p(q_out), _p(k_out), int(ranks),
            _handle(stream, dev))
    return q_out, k_out


def select_scratch_bytes(B: int, H: int, N: int, d: int) -> int:
    return int(sage.LIB.sage_select_scratch_bytes(B, H, N, d))


def alloc_select_scratch(B: int, H: int, N: int, d: int, device=None):
    """Scratch of select_blocks; calls that may overlap on the GPU need one each."""
    n = select_scratch_bytes(B, H, N, d)
    if n == 0:
        raise SageError(EINVAL, "sage_select_scratch_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def select_blocks(q, k, keep: int, first: int = 0, window: int = 0, lists=None, counts=None, scratch=None, stream=None):
    """The `keep` key blocks of every 128-token query block by the scores of pooled queries and keys
    (q, k bf16 [B, H, N, d]); blocks j < first and |i - j| <= window always (window -1: none).
    Returns (lists int32 [B, H, nT, keep] ascending with -1 behind, counts int32 [B, H, nT])."""
    B, H, N, d = sage._bhnd(q, "q")
    _is(q, "q", torch.bfloat16, q.shape)
    _is(k, "k", torch.bfloat16, q.shape)
    if keep < 1:
        raise ValueError("keep must be at least 1")
    nT = (N + BLK - 1) // BLK
    _is(lists, "lists", torch.int32, (B, H, nT, keep), optional=True)
    _is(counts, "counts", torch.int32, (B, H, nT), optional=True)
    _need(scratch, "scratch", torch.uint8, optional=True)
    dev = _where(stream, "q k lists counts scratch", q, k, lists, counts, scratch)
    if scratch is None:
        scratch = _new(q, max(select_scratch_bytes(B, H, N, d), 16), torch.uint8, stream)
    if lists is None:
        lists = _new(q, (B, H, nT, keep), torch.int32, stream)
    if counts is None:
        counts = _new(q, (B, H, nT), torch.int32, stream)
    _launch("sage_select_blocks", dev, _p(q), _p(k), B, H, N, d, int(keep), int(first), int(window), _p(lists),
            _p(counts), _p(scratch), scratch.numel(), _handle(stream, dev))
    return lists, counts


def _sparse_args(q, k, v, o, lists, counts, workspace):
    B, H, N, d = shape = tuple(sage._bhnd(q, "q"))
    _is(q, "q", torch.bfloat16, shape)
    _is(k, "k", torch.bfloat16, shape)
    _is(v, "v", torch.bfloat16, shape)
    _is(o, "o", torch.bfloat16, shape, optional=True)
    nT = (N + BLK - 1) // BLK
    _need(lists, "lists", torch.int32)
    if lists.dim() != 4 or lists.shape[3] < 1 or tuple(lists.shape[:3]) != (B, H, nT):
        raise ValueError(f"lists must have shape {(B, H, nT)} + (width,), got {tuple(lists.shape)}")
    _is(counts, "counts", torch.int32, (B, H, nT))
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return B, H, N, d


def attn_fwd_sparse(q, k, v, mode: int, lists, counts, coeff: int = COEFF_DIVIDE, o=None, workspace=None, stream=None):
    """Attention over the listed key blocks through sage_attn_fwd_sparse; returns bf16 O [B, H, N, d].

    lists int32 [B, H, nT, width], counts int32 [B, H, nT] as select_blocks gives them, or any lists: an empty
    one gives rows of 0.  coeff: how the INT8/FP8 modes round the quantization coefficients, COEFF_DIVIDE (the
    codes of the dense call) or COEFF_RECIPROCAL (the codes of torch's 127.0 / amax on the GPU).
    workspace: sage.alloc_workspace(B, H, N, d, mode); sage.status() on it reports a bad index or count (EINVAL),
    and calls that overlap on the GPU, in BF16 mode too, need one each.
    """
    B, H, N, d = _sparse_args(q, k, v, o, lists, counts, workspace)
    dev = _where(stream, "q k v o lists counts workspace", q, k, v, o, lists, counts, workspace)
    if o is None:
        o = _new(q, (B, H, N, d), torch.bfloat16, stream)
    if workspace is None:
        n = sage.workspace_bytes(B, H, N, d, mode)
        if n == 0:
            raise SageError(EINVAL, "sage_workspace_bytes")
        workspace = _new(q, n, torch.uint8, stream, zeroed=256)       # the status words
    _launch("sage_attn_fwd_sparse", dev, _p(q), _p(k), _p(v), _p(o), B, H, N, d, int(mode), _p(lists),
            _p(counts), lists.shape[3], int(coeff), _p(workspace), workspace.numel() * workspace.element_size(), _handle(stream, dev))
    return o


def dbg_sparse_forced_timeout(q, k, v, mode: int, lists, counts, workspace, timeout_cycles: int, stream=None):
    B, H, N, d = _sparse_args(q, k, v, None, lists, counts, workspace)
    dev = _where(stream, "q k v lists counts workspace", q, k, v, lists, counts, workspace)
    o = _new(q, (B, H, N, d), torch.bfloat16, stream)
    _launch("sage_dbg_sparse_forced_timeout", dev, _p(q), _p(k), _p(v), _p(o), B, H, N, d, int(mode),
            _p(lists), _p(counts), lists.shape[3], COEFF_DIVIDE, _p(workspace), workspace.numel() * workspace.element_size(),
            int(timeout_cycles), _handle(stream, dev))
    return o
