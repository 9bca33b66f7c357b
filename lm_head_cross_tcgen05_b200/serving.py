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
import functools

import torch

from . import (DTYPE_BF16, DTYPE_F32, ENTRY_FP8_LOGITS, ENTRY_RMS_NORM_BWD, ENTRY_SAMPLE, _bf, _f32,
               _i32, _ok, _u8, lmh_sampling, lmh_shape, lmh_workspace_size, make_shape)
from ._abi import lib

__all__ = ["lmh_rms_norm", "lmh_rms_norm_bwd", "lmh_quantize_fp8", "lmh_fp8_logits", "lmh_sample",
           "make_sampling", "rms_norm", "rms_norm_bwd", "quantize_fp8", "fp8_logits", "sample",
           "next_tokens"]

_e4m3 = torch.float8_e4m3fn
QBLOCK = 128  # columns (and, for a weight, rows) per scale


_DTYPES = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}


def _blocks(n: int) -> int:
    return -(-int(n) // QBLOCK)


def _shape_error(what, shape, t):
    return ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _arg(t, shape, dtype, what: str, dev: int):
    """The address of t (None stays None) after the checks: exactly this shape and type,
    contiguous, on device dev. Decode steps are a few microseconds of GPU time, so the checks
    are kept to what costs little on the host."""
    if t is None:
        return None
    if t.shape != shape:
        raise _shape_error(what, shape, t)
    if t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{what} is on {t.device}, another tensor of the call on device {dev}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def _own(t):
    """The address of a tensor that a helper has just made, which needs no checks."""
    return None if t is None else t.data_ptr()


def _matrix(t, what: str):
    if t.dim() != 2:
        raise ValueError(f"{what} must be a matrix, got {t.dim()} dimensions")
    return t.shape


_fns = {}


def _call(name: str, dev: int, stream, *args) -> None:
    """The entry with device dev current, on its current stream or on `stream`."""
    if dev < 0:
        raise ValueError(f"{name}: its tensors must be CUDA tensors")
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(dev)
    elif hasattr(stream, "cuda_stream"):
        if stream.device_index != dev:
            raise ValueError(f"{name}: a stream of device {stream.device_index} for tensors on {dev}")
        raw = stream.cuda_stream
    else:
        raw = int(stream)
    f = _fns.get(name)
    if f is None:
        f = _fns[name] = getattr(lib(), name)
    if dev == torch._C._cuda_getDevice():
        st = f(*args, raw)
    else:
        with torch.cuda.device(dev):
            st = f(*args, raw)
    if st != 0:
        _ok(name, st)


_here = contextlib.nullcontext()


def _allocating(stream, device):
    """Outputs of a helper belong to the stream that writes them."""
    if stream is None:
        return _here
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    return torch.cuda.stream(stream)


@functools.lru_cache(maxsize=4096)
def _ws_bytes(entry: int, N: int, d: int, V: int) -> int:
    n = lmh_workspace_size(make_shape(N, d, V), entry)
    if n == 0:
        raise ValueError("invalid shape for this entry")
    return n


def lmh_rms_norm(x, weight, residual=None, *, eps, sum=None, y=None, q=None, scale=None,
                 rstd=None, stream=None) -> None:
    N, d = _matrix(x, "x")
    dev, full = x.get_device(), (N, d)
    _call("lmh_rms_norm", dev, stream, N, d, _arg(x, full, _bf, "x", dev),
          _arg(residual, full, _bf, "residual", dev), _arg(weight, (d,), _bf, "weight", dev), eps,
          _arg(sum, full, _bf, "sum", dev), _arg(y, full, _bf, "y", dev),
          _arg(q, full, _e4m3, "q", dev), _arg(scale, (N, _blocks(d)), _f32, "scale", dev),
          _arg(rstd, (N,), _f32, "rstd", dev))


def lmh_rms_norm_bwd(sum, weight, rstd, dy, dsum=None, dx=None, dweight=None, *, workspace,
                     stream=None) -> None:
    N, d = _matrix(sum, "sum")
    dev, full = sum.get_device(), (N, d)
    _call("lmh_rms_norm_bwd", dev, stream, N, d, _arg(sum, full, _bf, "sum", dev),
          _arg(weight, (d,), _bf, "weight", dev), _arg(rstd, (N,), _f32, "rstd", dev),
          _arg(dy, full, _bf, "dy", dev), _arg(dsum, full, _bf, "dsum", dev),
          _arg(dx, full, _bf, "dx", dev), _arg(dweight, (d,), _bf, "dweight", dev),
          *_space(workspace, dev))


def lmh_quantize_fp8(x, q, scale, block_rows: int, *, stream=None) -> None:
    rows, d = _matrix(x, "x")
    if block_rows not in (1, QBLOCK):
        raise ValueError(f"block_rows must be 1 or {QBLOCK}, got {block_rows}")
    dev, full = x.get_device(), (rows, d)
    _call("lmh_quantize_fp8", dev, stream, rows, d, int(block_rows), _arg(x, full, _bf, "x", dev),
          _arg(q, full, _e4m3, "q", dev),
          _arg(scale, (-(-rows // block_rows), _blocks(d)), _f32, "scale", dev))


def _logits_dtype(t) -> int:
    if t not in _DTYPES:
        raise ValueError(f"logits must be torch.float32 or torch.bfloat16, got {t}")
    return _DTYPES[t]


def lmh_fp8_logits(shape, H8, h_scale, W8, w_scale, logits, *, workspace, stream=None) -> None:
    N, d, V, dev = shape.N, shape.d, shape.V, H8.get_device()
    nb, dt = _blocks(d), logits.dtype
    _call("lmh_fp8_logits", dev, stream, ctypes.byref(shape), _arg(H8, (N, d), _e4m3, "H8", dev),
          _arg(h_scale, (N, nb), _f32, "h_scale", dev), _arg(W8, (V, d), _e4m3, "W8", dev),
          _arg(w_scale, (_blocks(V), nb), _f32, "w_scale", dev),
          _arg(logits, (N, V), dt, "logits", dev), _logits_dtype(dt), *_space(workspace, dev))


def _space(workspace, dev: int):
    """(address, bytes) of a workspace."""
    return _arg(workspace, (workspace.numel(),), _u8, "workspace", dev), workspace.numel()


def make_sampling(N: int, top_k=None, top_p=None, min_p=None) -> lmh_sampling:
    """Each of top_k, top_p and min_p: None (off), a number for every row, or a CUDA tensor [N]
    (int32 for top_k, float32 for the others; kept alive by the caller for the call)."""
    o = lmh_sampling(0, 1.0, 0.0, None, None, None)
    if top_k is not None:
        if isinstance(top_k, torch.Tensor):
            o.row_top_k = _row_arg(top_k, N, _i32, "top_k")
        else:
            o.top_k = min(max(int(top_k), 0), 2 ** 31 - 1)
    if top_p is not None:
        if isinstance(top_p, torch.Tensor):
            o.row_top_p = _row_arg(top_p, N, _f32, "top_p")
        else:
            o.top_p = top_p
    if min_p is not None:
        if isinstance(min_p, torch.Tensor):
            o.row_min_p = _row_arg(min_p, N, _f32, "min_p")
        else:
            o.min_p = min_p
    return o


def _row_arg(t, N: int, dtype, what: str):
    at = _arg(t, (N,), dtype, what, t.get_device())
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    return at


def _same_device(t, dev: int) -> None:
    if t.get_device() != dev:
        raise ValueError(f"a row parameter is on {t.device}, the logits on device {dev}")


def lmh_sample(shape, opt, logits, u, tokens, logprob=None, *, workspace, stream=None,
               row_tensors=()) -> None:
    """row_tensors: the tensors that shape and opt point to, checked to be on the same device."""
    N, V, dev, dt = shape.N, shape.V, logits.get_device(), logits.dtype
    for t in row_tensors:
        _same_device(t, dev)
    _call("lmh_sample", dev, stream, ctypes.byref(shape), ctypes.byref(opt),
          _arg(logits, (N, V), dt, "logits", dev), _logits_dtype(dt), _arg(u, (N,), _f32, "u", dev),
          _arg(tokens, (N,), _i32, "tokens", dev), _arg(logprob, (N,), _f32, "logprob", dev),
          *_space(workspace, dev))


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
            out["y"] = torch.empty_like(x)
            out["rstd"] = torch.empty(N, dtype=_f32, device=dev)
        new = keep_sum and residual is not None
        out["sum"] = torch.empty_like(x) if new else None
    at, full, get = x.get_device(), (N, d), out.get
    _call("lmh_rms_norm", at, stream, N, d, _arg(x, full, _bf, "x", at),
          _arg(residual, full, _bf, "residual", at), _arg(weight, (d,), _bf, "weight", at), eps,
          _own(out["sum"]), _own(get("y")), _own(get("q")), _own(get("scale")), _own(get("rstd")))
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
        out = dict(dx=torch.empty_like(sum) if want_dx else None,
                   dweight=torch.empty(d, dtype=_bf, device=dev) if want_dweight else None)
        if ws is None:
            ws = torch.empty(_ws_bytes(ENTRY_RMS_NORM_BWD, N, d, 1), dtype=_u8, device=dev)
    at, full = sum.get_device(), (N, d)
    _call("lmh_rms_norm_bwd", at, stream, N, d, _arg(sum, full, _bf, "sum", at),
          _arg(weight, (d,), _bf, "weight", at), _arg(rstd, (N,), _f32, "rstd", at),
          _arg(dy, full, _bf, "dy", at), _arg(dsum, full, _bf, "dsum", at), _own(out["dx"]),
          _own(out["dweight"]), *_space(ws, at))
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
    dt, nb = _logits_dtype(dtype), _blocks(d)
    shape, dev = lmh_shape(N, d, V, 0, 0, 0, 0.0, None), H8.device
    with _allocating(stream, dev):
        out = dict(logits=torch.empty(N, V, dtype=dtype, device=dev))
        if ws is None:
            ws = torch.empty(_ws_bytes(ENTRY_FP8_LOGITS, N, d, V), dtype=_u8, device=dev)
    at = H8.get_device()
    _call("lmh_fp8_logits", at, stream, ctypes.byref(shape), _arg(H8, (N, d), _e4m3, "H8", at),
          _arg(h_scale, (N, nb), _f32, "h_scale", at), _arg(W8, (V, d), _e4m3, "W8", at),
          _arg(w_scale, (_blocks(V), nb), _f32, "w_scale", at), _own(out["logits"]), dt,
          *_space(ws, at))
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
    dt = _logits_dtype(logits.dtype)
    shape, dev = make_shape(N, 64, V, temperature=temperature), logits.device
    opt = make_sampling(N, top_k, top_p, min_p)
    with _allocating(stream, dev):
        out = dict(tokens=torch.empty(N, dtype=_i32, device=dev),
                   logprob=torch.empty(N, dtype=_f32, device=dev))
        if ws is None:
            ws = torch.empty(_ws_bytes(ENTRY_SAMPLE, N, 64, V), dtype=_u8, device=dev)
    at = logits.get_device()
    for t in (temperature, top_k, top_p, min_p):
        if isinstance(t, torch.Tensor):
            _same_device(t, at)
    _call("lmh_sample", at, stream, ctypes.byref(shape), ctypes.byref(opt),
          _arg(logits, (N, V), logits.dtype, "logits", at), dt, _arg(u, (N,), _f32, "u", at),
          _own(out["tokens"]), _own(out["logprob"]), *_space(ws, at))
    out["workspace"] = ws
    return out


def next_tokens(x, norm_weight, W8, w_scale, u, residual=None, *, eps: float = 1e-6,
                temperature=None, top_k=None, top_p=None, min_p=None, stream=None) -> dict:
    """The end of a decode step: the final RMS norm of x + residual into 8 bits, the 8-bit logits
    of the head (W8, w_scale from ``quantize_fp8``) and one token per row. The parameters are
    those of ``rms_norm`` and ``sample``; returns ``tokens``, ``logprob`` and ``logits``, with the
    two workspaces (``workspace`` of the sampling) for ``lmh_read_errors``."""
    n = rms_norm(x, norm_weight, residual, eps=eps, fp8=True, keep_sum=False, stream=stream)
    z = fp8_logits(n["q"], n["scale"], W8, w_scale, stream=stream)
    out = sample(z["logits"], u, temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p,
                 stream=stream)
    out["logits"], out["logits_workspace"] = z["logits"], z["workspace"]
    return out
