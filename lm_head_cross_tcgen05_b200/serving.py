"""The entries around the head: the RMS norm that makes its input (with its backward pass) and the
8-bit quantisation of both operands, the 8-bit logits, and the token drawn from logits;
``next_tokens`` is a decode step's end made of them.

As in the package's root, ``lmh_*`` mirror the C ABI on tensors that the caller allocated, and the
lower-case helpers allocate the outputs. All tensors of a call are on one CUDA device, which need
not be the current one; the work runs on that device's current stream, or on ``stream``, on which
a helper then allocates its outputs too. Nothing synchronises the host.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import (DTYPE_BF16, DTYPE_F32, ENTRY_FP8_LOGITS, ENTRY_RMS_NORM_BWD, ENTRY_SAMPLE, _bf, _f32,
               _i32, _ok, _p, _u8, lmh_sampling, lmh_workspace_size, make_shape)
from ._abi import lib

__all__ = ["lmh_rms_norm", "lmh_rms_norm_bwd", "lmh_quantize_fp8", "lmh_fp8_logits", "lmh_sample",
           "make_sampling", "rms_norm", "rms_norm_bwd", "quantize_fp8", "fp8_logits", "sample",
           "next_tokens"]

_e4m3 = torch.float8_e4m3fn
QBLOCK = 128  # columns (and, for a weight, rows) per scale


_DTYPES = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}


def _blocks(n: int) -> int:
    return -(-int(n) // QBLOCK)


def _shaped(**named) -> None:
    """Each named (tensor, shape): the tensor, when given, has exactly that shape."""
    for what, (t, shape) in named.items():
        if t is not None and tuple(t.shape) != tuple(shape):
            raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _matrix(t, what: str):
    if t.dim() != 2:
        raise ValueError(f"{what} must be a matrix, got {t.dim()} dimensions")
    return t.shape


def _call(name: str, tensors, stream, *args) -> None:
    """lib().name(*args, stream) with the tensors' device current."""
    dev = None
    for t in tensors:
        if t is not None:
            if dev is not None and t.device != dev:
                raise ValueError(f"{name}: tensors on {dev} and {t.device}")
            dev = t.device
    if stream is None:
        raw = torch.cuda.current_stream(dev).cuda_stream
    elif hasattr(stream, "cuda_stream"):
        if stream.device != dev:
            raise ValueError(f"{name}: a stream of {stream.device} for tensors on {dev}")
        raw = stream.cuda_stream
    else:
        raw = int(stream)
    f = getattr(lib(), name)
    if dev.index == torch.cuda.current_device():
        st = f(*args, raw)
    else:
        with torch.cuda.device(dev):
            st = f(*args, raw)
    _ok(name, st)


def _allocating(stream, device):
    """Outputs of a helper belong to the stream that writes them."""
    if stream is None:
        return contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    return torch.cuda.stream(stream)


def lmh_rms_norm(x, weight, residual=None, *, eps, sum=None, y=None, q=None, scale=None,
                 rstd=None, stream=None) -> None:
    N, d = _matrix(x, "x")
    _shaped(weight=(weight, (d,)), residual=(residual, (N, d)), sum=(sum, (N, d)), y=(y, (N, d)),
            q=(q, (N, d)), scale=(scale, (N, _blocks(d))), rstd=(rstd, (N,)))
    _call("lmh_rms_norm", (x, weight, residual, sum, y, q, scale, rstd), stream, N, d,
          _p(x, _bf, "x"), _p(residual, _bf, "residual"), _p(weight, _bf, "weight"), float(eps),
          _p(sum, _bf, "sum"), _p(y, _bf, "y"), _p(q, _e4m3, "q"), _p(scale, _f32, "scale"),
          _p(rstd, _f32, "rstd"))


def lmh_rms_norm_bwd(sum, weight, rstd, dy, dsum=None, dx=None, dweight=None, *, workspace,
                     stream=None) -> None:
    N, d = _matrix(sum, "sum")
    _shaped(weight=(weight, (d,)), rstd=(rstd, (N,)), dy=(dy, (N, d)), dsum=(dsum, (N, d)),
            dx=(dx, (N, d)), dweight=(dweight, (d,)))
    _call("lmh_rms_norm_bwd", (sum, weight, rstd, dy, dsum, dx, dweight, workspace), stream, N, d,
          _p(sum, _bf, "sum"), _p(weight, _bf, "weight"), _p(rstd, _f32, "rstd"),
          _p(dy, _bf, "dy"), _p(dsum, _bf, "dsum"), _p(dx, _bf, "dx"),
          _p(dweight, _bf, "dweight"), _p(workspace, _u8, "workspace"), workspace.numel())


def lmh_quantize_fp8(x, q, scale, block_rows: int, *, stream=None) -> None:
    rows, d = _matrix(x, "x")
    if block_rows not in (1, QBLOCK):
        raise ValueError(f"block_rows must be 1 or {QBLOCK}, got {block_rows}")
    _shaped(q=(q, (rows, d)), scale=(scale, (-(-rows // block_rows), _blocks(d))))
    _call("lmh_quantize_fp8", (x, q, scale), stream, rows, d, int(block_rows), _p(x, _bf, "x"),
          _p(q, _e4m3, "q"), _p(scale, _f32, "scale"))


def _logits_dtype(t) -> int:
    if t not in _DTYPES:
        raise ValueError(f"logits must be torch.float32 or torch.bfloat16, got {t}")
    return _DTYPES[t]


def lmh_fp8_logits(shape, H8, h_scale, W8, w_scale, logits, *, workspace, stream=None) -> None:
    N, d, V = shape.N, shape.d, shape.V
    _shaped(H8=(H8, (N, d)), h_scale=(h_scale, (N, _blocks(d))), W8=(W8, (V, d)),
            w_scale=(w_scale, (_blocks(V), _blocks(d))), logits=(logits, (N, V)))
    _call("lmh_fp8_logits", (H8, h_scale, W8, w_scale, logits, workspace), stream,
          ctypes.byref(shape), _p(H8, _e4m3, "H8"), _p(h_scale, _f32, "h_scale"),
          _p(W8, _e4m3, "W8"), _p(w_scale, _f32, "w_scale"), _p(logits, None, "logits"),
          _logits_dtype(logits.dtype), _p(workspace, _u8, "workspace"), workspace.numel())


def make_sampling(N: int, top_k=None, top_p=None, min_p=None) -> lmh_sampling:
    """Each of top_k, top_p and min_p: None (off), a number for every row, or a CUDA tensor [N]
    (int32 for top_k, float32 for the others; kept alive by the caller for the call)."""
    def rows(v, dtype, what):
        if not isinstance(v, torch.Tensor):
            return None
        _shaped(**{what: (v, (N,))})
        return _p(v, dtype, what)

    def scalar(v, off):
        return off if v is None or isinstance(v, torch.Tensor) else v
    k = min(max(int(scalar(top_k, 0)), 0), 2 ** 31 - 1)
    return lmh_sampling(k, float(scalar(top_p, 1.0)), float(scalar(min_p, 0.0)),
                        rows(top_k, _i32, "top_k"), rows(top_p, _f32, "top_p"),
                        rows(min_p, _f32, "min_p"))


def lmh_sample(shape, opt, logits, u, tokens, logprob=None, *, workspace, stream=None,
               row_tensors=()) -> None:
    """row_tensors: the tensors that shape and opt point to, checked to be on the same device."""
    N, V = shape.N, shape.V
    _shaped(logits=(logits, (N, V)), u=(u, (N,)), tokens=(tokens, (N,)), logprob=(logprob, (N,)))
    _call("lmh_sample", (logits, u, tokens, logprob, workspace, *row_tensors), stream,
          ctypes.byref(shape), ctypes.byref(opt), _p(logits, None, "logits"),
          _logits_dtype(logits.dtype), _p(u, _f32, "u"), _p(tokens, _i32, "tokens"),
          _p(logprob, _f32, "logprob"), _p(workspace, _u8, "workspace"), workspace.numel())


def rms_norm(x, weight, residual=None, *, eps: float = 1e-6, fp8: bool = False,
             keep_sum: bool = True, stream=None) -> dict:
    """The RMS norm of x + residual over rows of d: ``y`` (bf16) with ``rstd`` for the backward
    pass, or with fp8=True ``q`` (e4m3) and ``scale`` [N, ceil(d / 128)]. ``sum``: the stream
    x + residual as bf16 (x itself without a residual; None with keep_sum=False)."""
    N, d = _matrix(x, "x")
    dev = x.device
    out = {}
    with _allocating(stream, dev):
        if fp8:
            out["q"] = torch.empty(N, d, dtype=_e4m3, device=dev)
            out["scale"] = torch.empty(N, _blocks(d), dtype=_f32, device=dev)
        else:
            out["y"] = torch.empty(N, d, dtype=_bf, device=dev)
            out["rstd"] = torch.empty(N, dtype=_f32, device=dev)
        new = keep_sum and residual is not None
        out["sum"] = torch.empty(N, d, dtype=_bf, device=dev) if new else None
    lmh_rms_norm(x, weight, residual, eps=eps, stream=stream, **out)
    if keep_sum and residual is None:
        out["sum"] = x
    return out


def rms_norm_bwd(sum, weight, rstd, dy, dsum=None, *, want_dx: bool = True,
                 want_dweight: bool = True, ws=None, stream=None) -> dict:
    """Gradients of rms_norm from its ``sum`` and ``rstd``: ``dx`` (of x and of residual alike;
    dsum is the gradient that reaches the sum itself) and ``dweight``, both bf16."""
    N, d = _matrix(sum, "sum")
    dev = sum.device
    with _allocating(stream, dev):
        out = dict(dx=torch.empty(N, d, dtype=_bf, device=dev) if want_dx else None,
                   dweight=torch.empty(d, dtype=_bf, device=dev) if want_dweight else None)
        if ws is None:
            n = lmh_workspace_size(make_shape(N, d, 1), ENTRY_RMS_NORM_BWD)
            if n == 0:
                raise ValueError("invalid shape for this entry")
            ws = torch.empty(n, dtype=_u8, device=dev)
    lmh_rms_norm_bwd(sum, weight, rstd, dy, dsum, out["dx"], out["dweight"], workspace=ws,
                     stream=stream)
    return out


def quantize_fp8(x, block_rows: int = QBLOCK, *, stream=None):
    """(q, scale): x [rows, d] bf16 as e4m3 with one fp32 scale per block of block_rows x 128
    (128 for a weight, laid out once; 1 for hidden states)."""
    rows, d = _matrix(x, "x")
    if block_rows not in (1, QBLOCK):
        raise ValueError(f"block_rows must be 1 or {QBLOCK}, got {block_rows}")
    with _allocating(stream, x.device):
        q = torch.empty(rows, d, dtype=_e4m3, device=x.device)
        scale = torch.empty(-(-rows // block_rows), _blocks(d), dtype=_f32, device=x.device)
    lmh_quantize_fp8(x, q, scale, block_rows, stream=stream)
    return q, scale


def fp8_logits(H8, h_scale, W8, w_scale, *, dtype=torch.float32, ws=None, stream=None) -> dict:
    """``logits`` [N, V] (float32 or bfloat16) of 8-bit hidden states [N, d] (scales per row and
    128 columns) and an 8-bit head weight [V, d] (scales per 128 x 128 block)."""
    N, d = _matrix(H8, "H8")
    V = _matrix(W8, "W8")[0]
    _logits_dtype(dtype)
    shape, dev = make_shape(N, d, V), H8.device
    with _allocating(stream, dev):
        out = dict(logits=torch.empty(N, V, dtype=dtype, device=dev))
        if ws is None:
            n = lmh_workspace_size(shape, ENTRY_FP8_LOGITS)
            if n == 0:
                raise ValueError("invalid shape for this entry")
            ws = torch.empty(n, dtype=_u8, device=dev)
    lmh_fp8_logits(shape, H8, h_scale, W8, w_scale, out["logits"], workspace=ws, stream=stream)
    out["workspace"] = ws
    return out


def sample(logits, u, *, temperature=None, top_k=None, top_p=None, min_p=None, ws=None,
           stream=None) -> dict:
    """One token per row of logits [N, V] (float32 or bfloat16; -inf: cannot be drawn) at the
    uniform numbers u [N] (float32 in [0, 1)): temperature, then top-k, then top-p, then min-p,
    each None, a number or a CUDA tensor [N]. ``tokens`` int32 and ``logprob`` float32, the
    token's log-probability at that temperature before the filters; -1 and 0 for a row with no
    logit above -inf or with a NaN or +inf."""
    N, V = _matrix(logits, "logits")
    _logits_dtype(logits.dtype)
    shape, dev = make_shape(N, 64, V, temperature=temperature), logits.device
    opt = make_sampling(N, top_k, top_p, min_p)
    with _allocating(stream, dev):
        out = dict(tokens=torch.empty(N, dtype=_i32, device=dev),
                   logprob=torch.empty(N, dtype=_f32, device=dev))
        if ws is None:
            n = lmh_workspace_size(shape, ENTRY_SAMPLE)
            if n == 0:
                raise ValueError("invalid shape for this entry")
            ws = torch.empty(n, dtype=_u8, device=dev)
    rows = [t for t in (temperature, top_k, top_p, min_p) if isinstance(t, torch.Tensor)]
    lmh_sample(shape, opt, logits, u, out["tokens"], out["logprob"], workspace=ws, stream=stream,
               row_tensors=rows)
    out["workspace"] = ws
    return out


def next_tokens(x, norm_weight, W8, w_scale, u, residual=None, *, eps: float = 1e-6,
                temperature=None, top_k=None, top_p=None, min_p=None, stream=None) -> dict:
    """The end of a decode step: the final RMS norm of x + residual into 8 bits, the 8-bit logits
    of the head (W8, w_scale from ``quantize_fp8``) and one token per row. The parameters are
    those of ``rms_norm`` and ``sample``; returns ``tokens``, ``logprob`` and ``logits``."""
    n = rms_norm(x, norm_weight, residual, eps=eps, fp8=True, keep_sum=False, stream=stream)
    z = fp8_logits(n["q"], n["scale"], W8, w_scale, stream=stream)
    out = sample(z["logits"], u, temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p,
                 stream=stream)
    out["logits"] = z["logits"]
    return out
