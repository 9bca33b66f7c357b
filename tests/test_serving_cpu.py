"""Refusals of the entries around the head, found on the host before any CUDA call (CPU)."""
import ctypes

import pytest
import torch

import lm_head_cross_tcgen05_b200 as L
from lm_head_cross_tcgen05_b200._abi import lib

INVALID, SHORT, ALIGN = 1, 3, 4
P = 4096  # a pointer that no refused call follows


def norm(N=1, d=64, x=P, residual=None, weight=P, eps=1e-6, sum=None, y=P, q=None, scale=None, rstd=None):
    return lib().lmh_rms_norm(N, d, x, residual, weight, eps, sum, y, q, scale, rstd, None)


@pytest.mark.parametrize("kw,status", [
    (dict(d=0), INVALID), (dict(d=96), INVALID), (dict(d=16448), INVALID), (dict(N=-1), INVALID), (dict(N=2 ** 31), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(y=None), INVALID), (dict(q=P), INVALID), (dict(scale=P), INVALID), (dict(x=None), INVALID), (dict(weight=None), INVALID),
    (dict(x=P + 2), ALIGN), (dict(residual=P + 8), ALIGN), (dict(y=P + 2), ALIGN), (dict(q=P + 8, scale=P), ALIGN),
    (dict(q=P, scale=P + 2), ALIGN), (dict(rstd=P + 1), ALIGN), (dict(sum=P + 4), ALIGN), (dict(weight=P + 2), ALIGN)])
def test_norm_refuses(kw, status):
    assert norm(**kw) == status


def norm_bwd(N=1, d=64, sum=P, weight=P, rstd=P, dy=P, dsum=None, dx=P, dweight=P, ws=P, n=1 << 20):
    return lib().lmh_rms_norm_bwd(N, d, sum, weight, rstd, dy, dsum, dx, dweight, ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(d=65), INVALID), (dict(N=-1), INVALID), (dict(dx=None, dweight=None), INVALID), (dict(ws=None), INVALID),
    (dict(sum=None), INVALID), (dict(dy=None), INVALID), (dict(rstd=None), INVALID), (dict(weight=None), INVALID),
    (dict(dsum=P + 2), ALIGN), (dict(ws=P + 16), ALIGN), (dict(rstd=P + 2), ALIGN), (dict(n=511), SHORT),
    (dict(N=10 ** 6, d=16384, n=148 * 16384 * 4), SHORT)])
def test_norm_bwd_refuses(kw, status):
    assert norm_bwd(**kw) == status


def test_norm_bwd_workspace():
    def ws(N, d):
        return L.lmh_workspace_size(L.make_shape(N, d, 1), L.ENTRY_RMS_NORM_BWD)
    assert ws(1, 64) == 512 and ws(0, 64) == 256
    assert ws(296, 4096) == ws(10 ** 6, 4096) == 256 + 296 * 4096 * 4 and ws(10 ** 6, 2048) == 256 + 592 * 2048 * 4
    assert ws(1, 16448) == 0 and ws(2 ** 31, 64) == 0


@pytest.mark.parametrize("args,status", [
    ((1, 96, 1, P, P, P), INVALID), ((-1, 64, 1, P, P, P), INVALID), ((1, 64, 64, P, P, P), INVALID), ((1, 64, 0, P, P, P), INVALID),
    ((1, 64, 1, None, P, P), INVALID), ((1, 64, 1, P, None, P), INVALID), ((1, 64, 1, P, P, None), INVALID),
    ((2 ** 31 - 1, 2 ** 24, 1, P, P, P), INVALID), ((1, 64, 1, P + 8, P, P), ALIGN), ((1, 64, 1, P, P + 8, P), ALIGN),
    ((1, 64, 1, P, P, P + 2), ALIGN)])
def test_quantize_refuses(args, status):
    assert lib().lmh_quantize_fp8(*args, None) == status


def test_python_refuses():
    b = torch.bfloat16
    x, w = torch.zeros(2, 64, dtype=b), torch.zeros(64, dtype=b)
    with pytest.raises(ValueError, match="matrix"):
        L.rms_norm(x[0], w)
    with pytest.raises(ValueError, match="weight must have shape"):
        L.rms_norm(x, w[:32])
    with pytest.raises(ValueError, match="residual must have shape"):
        L.rms_norm(x, w, x[:1])
    with pytest.raises(ValueError, match="CUDA"):
        L.rms_norm(x, w)
    with pytest.raises(ValueError, match="block_rows"):
        L.quantize_fp8(x, 64)
    with pytest.raises(ValueError, match="rstd must have shape"):
        L.rms_norm_bwd(x, w, torch.zeros(3), x)


def logits(N=1, V=100, d=64, H8=P, hs=P, W8=P, ws=P, out=P, dtype=0, work=P, n=1 << 20):
    shape = L.make_shape(N, d, V)
    return lib().lmh_fp8_logits(ctypes.byref(shape), H8, hs, W8, ws, out, dtype, work, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(d=32), INVALID), (dict(V=0), INVALID), (dict(N=-1), INVALID), (dict(N=2 ** 31), INVALID), (dict(dtype=2), INVALID),
    (dict(dtype=-1), INVALID), (dict(H8=None), INVALID), (dict(hs=None), INVALID), (dict(W8=None), INVALID), (dict(ws=None), INVALID),
    (dict(out=None), INVALID), (dict(work=None), INVALID), (dict(H8=P + 8), ALIGN), (dict(W8=P + 8), ALIGN), (dict(hs=P + 2), ALIGN),
    (dict(out=P + 2), ALIGN), (dict(out=P + 1, dtype=1), ALIGN), (dict(work=P + 128), ALIGN), (dict(n=255), SHORT)])
def test_logits_refuses(kw, status):
    assert logits(**kw) == status


def test_logits_python_refuses():
    e4 = torch.float8_e4m3fn
    H, W = torch.zeros(2, 192).to(e4), torch.zeros(130, 192).to(e4)
    hs, ws = torch.ones(2, 2), torch.ones(2, 2)
    with pytest.raises(ValueError, match="CUDA"):
        L.lmh_fp8_logits(L.make_shape(2, 192, 130), H, hs, W, ws, torch.zeros(2, 130), workspace=torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(ValueError, match="w_scale must have shape"):
        L.lmh_fp8_logits(L.make_shape(2, 192, 130), H, hs, W, torch.ones(2, 1), torch.zeros(2, 130), workspace=torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(ValueError, match="logits must be"):
        L.fp8_logits(H, hs, W, ws, dtype=torch.float16)


def sample(N=1, V=100, logits=P, dtype=0, u=P, tokens=P, logprob=None, work=P, n=1 << 20, tau=None, no_opt=False, **kw):
    shape = L.make_shape(N, 64, V, temperature=tau)
    o = L.make_sampling(N, **kw)
    return lib().lmh_sample(ctypes.byref(shape), None if no_opt else ctypes.byref(o), logits, dtype, u, tokens, logprob, work, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(V=0), INVALID), (dict(V=2 ** 31), INVALID), (dict(N=-1), INVALID), (dict(N=2 ** 28), INVALID), (dict(dtype=3), INVALID),
    (dict(logits=None), INVALID), (dict(u=None), INVALID), (dict(tokens=None), INVALID), (dict(work=None), INVALID),
    (dict(top_p=float("nan")), INVALID), (dict(min_p=float("nan")), INVALID), (dict(tau=float("nan")), INVALID), (dict(tau=-1.0), INVALID),
    (dict(no_opt=True), INVALID), (dict(logits=P + 2), ALIGN), (dict(logits=P + 1, dtype=1), ALIGN), (dict(u=P + 2), ALIGN),
    (dict(tokens=P + 2), ALIGN), (dict(logprob=P + 2), ALIGN), (dict(work=P + 4), ALIGN), (dict(n=128), SHORT)])
def test_sample_refuses(kw, status):
    assert sample(**kw) == status


def test_sample_python_refuses():
    z, u = torch.zeros(2, 10), torch.zeros(2)
    with pytest.raises(ValueError, match="CUDA"):
        L.sample(z, u, top_k=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="top_p must have shape"):
        L.make_sampling(2, top_p=torch.ones(3))
    with pytest.raises(ValueError, match="logits must be"):
        L.sample(z.half(), u)
    with pytest.raises(ValueError, match="u must have shape"):
        L.lmh_sample(L.make_shape(2, 64, 10), L.make_sampling(2), z, torch.zeros(3), torch.zeros(2, dtype=torch.int32),
                     workspace=torch.zeros(256, dtype=torch.uint8))
