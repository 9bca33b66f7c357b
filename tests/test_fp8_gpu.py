"""8-bit logits against the fp64 oracle on the same 8-bit values and scales.

Tolerance. Products of two e4m3 values are exact in fp32. A block's 128 products are added on the
tensor core, whose additions may truncate: at most one step (2^-23) of a partial sum each. The
block's scale (a product of two numbers, 2^-24) is applied with one fused multiply-add per block
(2^-24 each, nb of them). All relative to the sum of the terms' magnitudes; the logit's own
rounding is 2^-24 (fp32) or 2^-8 (bf16) of it."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import lm_head_cross_tcgen05_b200 as L
from oracle import serving_oracle as S

pytestmark = pytest.mark.gpu


def f64(t):
    return t.detach().cpu().double().numpy()


def operands(N, V, d, seed=0, wild=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    H = torch.randn(N, d, device="cuda", generator=g)
    W = torch.randn(V, d, device="cuda", generator=g) * 0.02
    if wild:  # blocks of very different scales
        H *= torch.exp(2 * torch.randn(N, 1, device="cuda", generator=g))
        W *= torch.exp(torch.randn(1, d, device="cuda", generator=g))
    return L.quantize_fp8(H.bfloat16(), 1) + L.quantize_fp8(W.bfloat16())


def check(z, H8, hs, W8, ws):
    h, w = f64(H8.float()), f64(W8.float())
    want = S.logits(h, f64(hs), w, f64(ws))
    mags = S.logits(np.abs(h), f64(hs), np.abs(w), f64(ws))
    e = (128 * 2.0 ** -23 + (hs.shape[1] + 1) * 2.0 ** -24) * mags
    own = 2.0 ** -8 if z.dtype == torch.bfloat16 else 2.0 ** -24
    assert np.all(np.abs(f64(z.float()) - want) <= e * (1 + own) + own * np.abs(want))


CASES = [(1, 1, 64), (1, 100, 128), (3, 127, 192), (16, 128, 64), (17, 129, 256), (32, 255, 320), (33, 257, 2112),
         (64, 1000, 512), (65, 1000, 512), (100, 128, 64), (128, 256, 128), (129, 257, 192), (300, 700, 1088), (1, 40000, 128),
         (2, 20000, 1024), (513, 3000, 256)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,V,d", CASES)
def test_logits(N, V, d, dtype):
    ops = operands(N, V, d, seed=N + V)
    o = L.fp8_logits(*ops, dtype=dtype)
    assert L.lmh_read_errors(o["workspace"]) == 0
    check(o["logits"], *ops)
    assert torch.equal(L.fp8_logits(*ops, dtype=dtype)["logits"], o["logits"])


@pytest.mark.parametrize("N", [1, 20, 64, 130])
def test_small_whole_numbers_are_exact(N):
    """Whole numbers below 2^24 in all partial sums, scales of powers of two: no rounding at all."""
    V, d = 391, 448
    g = torch.Generator(device="cuda").manual_seed(N)
    h = torch.randint(-8, 9, (N, d), device="cuda", generator=g).float()
    w = torch.randint(-8, 9, (V, d), device="cuda", generator=g).float()
    hs = 2.0 ** torch.randint(-3, 4, (N, 4), device="cuda", generator=g).float()
    ws = 2.0 ** torch.randint(-3, 4, (4, 4), device="cuda", generator=g).float()
    z = L.fp8_logits(h.to(torch.float8_e4m3fn), hs, w.to(torch.float8_e4m3fn), ws)["logits"]
    assert np.array_equal(f64(z), S.logits(f64(h), f64(hs), f64(w), f64(ws)))


@pytest.mark.parametrize("N", [5, 90])
def test_largest_values_and_nan(N):
    V, d = 300, 256
    h = torch.full((N, d), 448.0, device="cuda")
    w = torch.full((V, d), -448.0, device="cuda")
    w[7, 130] = float("nan")
    h[2, 5] = float("nan")
    hs, ws = torch.ones(N, 2, device="cuda"), torch.ones(3, 2, device="cuda")
    z = L.fp8_logits(h.to(torch.float8_e4m3fn), hs, w.to(torch.float8_e4m3fn), ws)["logits"]
    bad = torch.isnan(z)
    assert torch.all(bad[2]) and torch.all(bad[:, 7]) and int(bad.sum()) == V + N - 1
    assert torch.all(z[~bad] == -448.0 * 448.0 * d)
    hs[0, 0] = float("inf")
    z = L.fp8_logits(h.to(torch.float8_e4m3fn), hs, w.to(torch.float8_e4m3fn), ws)["logits"]
    assert torch.all(torch.isinf(z[0, :7]))


def test_nothing_is_written_beside_the_logits():
    N, V, d = 70, 333, 192
    ops = operands(N, V, d, seed=3)
    for dtype in (torch.float32, torch.bfloat16):
        for n in (13, N):
            room = torch.full((n * V + 512,), 7.0, device="cuda", dtype=dtype)
            z = room[256:256 + n * V].view(n, V)
            shape = L.make_shape(n, d, V)
            ws = torch.empty(L.lmh_workspace_size(shape, L.ENTRY_FP8_LOGITS), dtype=torch.uint8, device="cuda")
            L.lmh_fp8_logits(shape, ops[0][:n], ops[1][:n], ops[2], ops[3], z, workspace=ws)
            assert torch.all(room[:256] == 7) and torch.all(room[256 + n * V:] == 7)
            assert torch.equal(z, L.fp8_logits(ops[0][:n], ops[1][:n], ops[2], ops[3], dtype=dtype)["logits"])


def test_offsets_past_32_bits():
    """More than 2^31 logits, and a weight of more than 2^31 bytes."""
    N, V, d = 1100, 2 ** 21, 1088
    g = torch.Generator(device="cuda").manual_seed(4)
    H8, hs = L.quantize_fp8(torch.randn(N, d, device="cuda", generator=g).bfloat16(), 1)
    W8 = torch.zeros(V, d, device="cuda", dtype=torch.uint8)
    tail = torch.randn(300, d, device="cuda", generator=g).to(torch.float8_e4m3fn)
    W8[-300:] = tail.view(torch.uint8)
    W8 = W8.view(torch.float8_e4m3fn)
    ws = torch.full((V // 128, 9), 0.25, device="cuda")
    z = L.fp8_logits(H8, hs, W8, ws, dtype=torch.bfloat16)["logits"]
    check(z[-3:, -300:], H8[-3:], hs[-3:], tail, ws[:3])
    assert float(z[:, :-300].abs().max()) == 0
    del z
    z = L.fp8_logits(H8[:1], hs[:1], W8, ws)["logits"]
    check(z[:, -300:], H8[:1], hs[:1], tail, ws[:3])


def test_no_rows():
    ops = operands(1, 100, 64)
    o = L.fp8_logits(ops[0][:0], ops[1][:0], ops[2], ops[3])
    assert o["logits"].shape == (0, 100) and L.lmh_read_errors(o["workspace"]) == 0


def test_another_stream_and_two_graphs():
    """Two captured graphs, each with its own workspace, and new inputs at the replay."""
    V, d = 900, 512
    a, b = operands(3, V, d, seed=5), operands(100, V, d, seed=6)
    L.fp8_logits(*a), L.fp8_logits(*b)
    graphs, outs = [], []
    for ops in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(L.fp8_logits(*ops)["logits"])
        graphs.append(g)
    for ops, seed in ((a, 7), (b, 8)):
        for t, new in zip(ops, operands(ops[0].shape[0], V, d, seed=seed)):
            t.view(torch.uint8).copy_(new.view(torch.uint8))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for g, s in zip(graphs, streams):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    for ops, z in ((a, outs[0]), (b, outs[1])):
        got = L.fp8_logits(*ops, stream=streams[0])["logits"]
        streams[0].synchronize()
        assert torch.equal(z, got)
        check(z, *ops)


@pytest.mark.parametrize("N", [3, 40, 70])
def test_long_rows(N):
    """More scale blocks than the few-token kernel keeps, and just as many."""
    for d in (8192, 8256, 16448):
        ops = operands(N, 260, d, seed=d)
        check(L.fp8_logits(*ops)["logits"], *ops)


def test_stale_error_word_is_cleared():
    ops = operands(2, 300, 128)
    shape = L.make_shape(2, 128, 300)
    ws = torch.full((L.lmh_workspace_size(shape, L.ENTRY_FP8_LOGITS),), 255, dtype=torch.uint8, device="cuda")
    L.fp8_logits(*ops, ws=ws)
    assert L.lmh_read_errors(ws) == 0


@pytest.mark.parametrize("N", [5, 130])
@pytest.mark.parametrize("d", [512, 576])
def test_scales_at_any_address(N, d):
    """Scales aligned to 4 bytes only, H8 and W8 to 16; the logits the same as from aligned ones."""
    ops = operands(N, 300, d, seed=9)
    moved = []
    for t, by in zip(ops, (16, 1, 16, 1)):
        flat = torch.zeros(t.numel() + by, dtype=t.dtype, device="cuda")
        flat[by:].copy_(t.flatten())
        moved.append(flat[by:].view(t.shape))
    assert torch.equal(L.fp8_logits(*moved)["logits"], L.fp8_logits(*ops)["logits"])


def test_two_calls_at_once():
    a, b = operands(40, 5000, 640, seed=10), operands(200, 5000, 640, seed=11)
    ref = [L.fp8_logits(*x)["logits"] for x in (a, b)]
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        z = [L.fp8_logits(*x, stream=t)["logits"] for x, t in zip((a, b), s)]
        torch.cuda.synchronize()
        assert torch.equal(z[0], ref[0]) and torch.equal(z[1], ref[1])
