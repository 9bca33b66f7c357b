"""RMS norm with residual (bf16 and e4m3 outputs), its backward pass and the e4m3 quantisation
against the fp64 oracle.

Tolerances. A rounding to a type is off by at most half a step: 2^-8 (bf16), 2^-4 (e4m3; 2^-10 of
the scale below its smallest normal value) of the value. fp32 steps before it: a thread adds at
most 32 squares, then 5 + 16 partial sums follow, all positive, so the sum of squares is off by
less than 56 * 2^-24 of itself and rstd by half of that plus 3 roundings: below 2^-18, which E32
allows for every fp32 quantity, relative to the sum of its terms' magnitudes."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import lm_head_cross_tcgen05_b200 as L
from lm_head_cross_tcgen05_b200 import autograd as A
from oracle import serving_oracle as S

pytestmark = pytest.mark.gpu

BF, E4, E32 = 2.0 ** -8, 2.0 ** -4, 2.0 ** -18
SHAPES = [(1, 64), (1, 4096), (2, 192), (3, 256), (5, 320), (7, 512), (33, 1344), (4, 4160), (3, 8192),
          (2, 8256), (3, 16384), (700, 128), (1500, 704)]


def f64(t):
    return t.detach().cpu().double().numpy()


def rand(*shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, device="cuda", generator=g) * scale).bfloat16()


def check_q(q, scale, y, block_rows, slack=E32):
    """q * scale against y, and the scales against those of y; slack: how far the quantised
    values may be from y before their rounding."""
    want = S.block_scales(y, block_rows)
    s = f64(scale)
    assert np.all(np.abs(s - want) <= (slack + 2.0 ** -24) * want)
    full = S.expand(s, block_rows, y.shape)
    got = f64(q.float()) * full
    assert np.all(np.abs(got - y) <= (E4 * (1 + slack) + 2 * slack) * np.abs(y) + 2.0 ** -10 * full)


@pytest.mark.parametrize("N,d", SHAPES)
@pytest.mark.parametrize("res", [False, True])
def test_forward(N, d, res):
    x, r, w = rand(N, d, seed=1, scale=3), rand(N, d, seed=2), rand(d, seed=3)
    r = r if res else None
    o = L.rms_norm(x, w, r, eps=1e-5)
    o8 = L.rms_norm(x, w, r, eps=1e-5, fp8=True)
    total = (x.float() + r.float()).bfloat16() if res else x
    assert torch.equal(o["sum"], total) and torch.equal(o8["sum"], total)
    y, rstd = S.rms_norm(f64(total), f64(w), 1e-5)
    assert np.all(np.abs(f64(o["rstd"]) - rstd) <= E32 * rstd)
    assert np.all(np.abs(f64(o["y"]) - y) <= (BF + E32) * np.abs(y))
    check_q(o8["q"], o8["scale"], y, 1)


@pytest.mark.parametrize("N,d", SHAPES)
def test_backward(N, d):
    x, w, dy, ds = rand(N, d, seed=4, scale=2), rand(d, seed=5), rand(N, d, seed=6, scale=1e-2), rand(N, d, seed=7, scale=1e-2)
    f = L.rms_norm(x, w, eps=1e-5)
    for dsum in (None, ds):
        b = L.rms_norm_bwd(f["sum"], w, f["rstd"], dy, dsum)
        r, wf, g = f64(x), f64(w), f64(dy)
        dx, dw = S.rms_norm_bwd(r, wf, 1e-5, g, None if dsum is None else f64(dsum))
        rstd = 1 / np.sqrt((r * r).mean(1, keepdims=True) + 1e-5)
        n = np.abs(r * rstd)
        terms = rstd * (np.abs(wf * g) + n * (np.abs(wf * g) * n).mean(1, keepdims=True))
        terms = terms + (0 if dsum is None else np.abs(f64(dsum)))
        # c's terms, added in at most 56 steps, are each off by rstd's error twice
        assert np.all(np.abs(f64(b["dx"]) - dx) <= BF * np.abs(dx) + 3 * E32 * terms)
        # dweight: at most ceil(N / 148) rows per slice, then every 16th of at most 2368 slices and
        # these 16 sums; rstd's error per term
        steps = -(-N // 148) + 148 + 16
        mags = (np.abs(g) * n).sum(0)
        assert np.all(np.abs(f64(b["dweight"]) - dw) <= BF * np.abs(dw) + (E32 + (steps + 2) * 2.0 ** -24) * mags)


def test_one_gradient_alone_and_in_place():
    N, d = 37, 320
    x, w, dy, ds = rand(N, d, seed=8), rand(d, seed=9), rand(N, d, seed=10), rand(N, d, seed=11)
    f = L.rms_norm(x, w)
    b = L.rms_norm_bwd(f["sum"], w, f["rstd"], dy, ds)
    assert torch.equal(L.rms_norm_bwd(f["sum"], w, f["rstd"], dy, ds, want_dx=False)["dweight"], b["dweight"])
    assert torch.equal(L.rms_norm_bwd(f["sum"], w, f["rstd"], dy, ds, want_dweight=False)["dx"], b["dx"])
    ws = torch.empty(L.lmh_workspace_size(L.make_shape(N, d, 1), L.ENTRY_RMS_NORM_BWD), dtype=torch.uint8, device="cuda")
    for into in (0, 1):
        a = [dy.clone(), ds.clone()]
        L.lmh_rms_norm_bwd(f["sum"], w, f["rstd"], a[0], a[1], dx=a[into], workspace=ws)
        assert torch.equal(a[into], b["dx"])
    assert L.lmh_read_errors(ws) == 0
    r = rand(N, d, seed=12)
    o = L.rms_norm(x, w, r)
    for k in (0, 1):
        a = [x.clone(), r.clone()]
        y = torch.empty_like(x)
        L.lmh_rms_norm(a[0], w, a[1], eps=1e-6, sum=a[k], y=y)
        assert torch.equal(a[k], o["sum"]) and torch.equal(y, o["y"])


def test_both_outputs_in_one_call():
    x, w = rand(5, 192, seed=13), rand(192, seed=14)
    y, q = torch.empty_like(x), torch.empty(5, 192, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(5, 2, device="cuda")
    L.lmh_rms_norm(x, w, eps=1e-6, y=y, q=q, scale=s)
    o, o8 = L.rms_norm(x, w), L.rms_norm(x, w, fp8=True)
    assert torch.equal(y, o["y"]) and torch.equal(q.view(torch.uint8), o8["q"].view(torch.uint8)) and torch.equal(s, o8["scale"])


def test_rows_of_zeros_infinities_and_nan():
    x, w = rand(5, 128, seed=15), torch.ones(128, device="cuda", dtype=torch.bfloat16)
    x[0] = 0
    x[1, 3] = float("inf")
    x[2, 3] = float("nan")
    x[3] = 1e-38
    o, o8 = L.rms_norm(x, w, eps=1e-6), L.rms_norm(x, w, eps=1e-6, fp8=True)
    y, q, s = o["y"].float(), o8["q"].float(), o8["scale"]
    assert torch.all(y[0] == 0) and torch.all(q[0] == 0) and float(s[0, 0]) == np.float32(2.0 ** -100 / 448)
    assert torch.isnan(y[1, 3]) and torch.all(torch.cat([y[1, :3], y[1, 4:]]) == 0) and torch.isnan(s[1, 0])
    assert torch.all(torch.isnan(y[2])) and torch.all(torch.isnan(q[2])) and torch.isnan(s[2, 0])
    assert np.allclose(f64(o["y"][3]), 1e-35, rtol=BF + 2.0 ** -8)  # 1e-38 is itself rounded to bf16
    ref = L.rms_norm(x[4:].clone(), w, eps=1e-6)
    assert torch.equal(ref["y"], o["y"][4:])  # a row does not see its neighbours


@pytest.mark.parametrize("rows,d,block_rows", [(1, 64, 1), (1, 64, 128), (127, 192, 128), (129, 128, 128), (300, 704, 1),
                                               (513, 2112, 128), (77, 16448, 1), (77, 16448, 128)])
def test_quantize(rows, d, block_rows):
    x = rand(rows, d, seed=16, scale=0.02)
    x[:, :64] *= 100
    x[0, 0] = 0
    q, s = L.quantize_fp8(x, block_rows)
    check_q(q, s, f64(x), block_rows, slack=2.0 ** -23)
    # every block's largest value is +-448
    full = S.expand(S.block_scales(f64(x), block_rows) * S.E4M3_MAX, block_rows, (rows, d))
    hit = np.abs(f64(x)) == full
    assert np.all(np.abs(f64(q.float()))[hit] == 448)


def test_quantize_special_blocks():
    x = torch.zeros(256, 256, device="cuda", dtype=torch.bfloat16)
    x[0, 128:] = 1.0
    x[130, 5] = float("nan")
    x[140, 200], x[141, 201] = float("-inf"), 2.0
    x[3, 3] = 1e-39  # a subnormal
    q, s = L.quantize_fp8(x)
    qf = q.float()
    assert float(s[0, 0]) == np.float32(2.0 ** -100 / 448) and torch.all(qf[:128, :128] == 0)
    assert torch.all(qf[0, 128:] == 448) and torch.all(qf[1:128, 128:] == 0)
    assert torch.isnan(s[1, 0]) and torch.all(torch.isnan(qf[128:, :128]))
    assert torch.isinf(s[1, 1]) and torch.isnan(qf[140, 200]) and float(qf[141, 201]) == 0


def test_no_rows():
    e = torch.empty(0, 128, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(128, device="cuda", dtype=torch.bfloat16)
    o = L.rms_norm(e, w, e)
    assert o["y"].shape == (0, 128)
    b = L.rms_norm_bwd(o["sum"], w, o["rstd"], e)
    assert b["dx"].shape == (0, 128) and torch.all(b["dweight"] == 0)
    q, s = L.quantize_fp8(e)
    assert q.shape == (0, 128) and s.shape == (0, 1)


def test_rows_past_32_bit_offsets():
    """More than 2^31 elements: the last rows are those of a small call."""
    d = 16384
    N = 2 ** 31 // d + 3
    x = torch.zeros(N, d, device="cuda", dtype=torch.bfloat16)
    x[-3:] = rand(3, d, seed=17)
    w = rand(d, seed=18)
    o = L.rms_norm(x, w, fp8=True)
    ref = L.rms_norm(x[-3:].clone(), w, fp8=True)
    assert torch.equal(o["q"][-3:].view(torch.uint8), ref["q"].view(torch.uint8)) and torch.equal(o["scale"][-3:], ref["scale"])
    for br in (1, 128):
        q, s = L.quantize_fp8(x, br)
        assert torch.all(q[:-3].view(torch.uint8)[::997] == 0)
        lo = (N - 3) // 128 * 128 if br == 128 else N - 3
        q2, s2 = L.quantize_fp8(x[lo:].clone(), br)
        assert torch.equal(q[lo:].view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s[-s2.shape[0]:], s2)


def test_autograd_and_the_head_behind_it():
    """rms_norm -> cross_entropy -> backward: the leaves' gradients are those of the entries."""
    N, d, V = 61, 192, 700
    x, r, w, W = rand(N, d, seed=19), rand(N, d, seed=20), rand(d, seed=21), rand(V, d, seed=22, scale=0.05)
    y = torch.randint(0, V, (N,), device="cuda", dtype=torch.int32)
    leaves = [t.clone().requires_grad_() for t in (x, r, w, W)]
    H, total = A.rms_norm(leaves[0], leaves[2], leaves[1])
    (A.cross_entropy(H, leaves[3], y) + 0.1 * total.float().square().mean()).backward()
    f = L.rms_norm(x, w, r)
    dsum = (0.2 * f["sum"].float() / (N * d)).bfloat16()
    g = L.loss_fwd(f["y"], W, y, grads=True)
    b = L.rms_norm_bwd(f["sum"], w, f["rstd"], g["dH"], dsum)
    assert torch.equal(leaves[3].grad, g["dW"]) and torch.equal(leaves[2].grad, b["dweight"])
    # 0.1 * grad of the mean square, formed by torch in another order: one bf16 step of dsum
    assert torch.equal(leaves[0].grad, leaves[1].grad)
    assert torch.all((leaves[0].grad.float() - b["dx"].float()).abs() <= 2 * BF * (b["dx"].float().abs() + dsum.float().abs()))


@pytest.mark.parametrize("res", [False, True])
def test_autograd_parts(res):
    N, d = 9, 128
    x, r, w, g = rand(N, d, seed=23), rand(N, d, seed=24), rand(d, seed=25), rand(N, d, seed=26)
    lx, lw, lr = x.clone().requires_grad_(), w.clone().requires_grad_(), r.clone().requires_grad_()
    out = A.rms_norm(lx, lw, lr if res else None)
    H = out[0] if res else out
    H.backward(g.t().contiguous().t() if d > 1 else g)  # an upstream gradient that is not contiguous
    f = L.rms_norm(x, w, r if res else None)
    b = L.rms_norm_bwd(f["sum"], w, f["rstd"], g)
    assert torch.equal(lx.grad, b["dx"]) and torch.equal(lw.grad, b["dweight"])
    if res:
        assert torch.equal(lr.grad, b["dx"])
        lx.grad = lr.grad = lw.grad = None  # only the sum is used
        _, total = A.rms_norm(lx, lw, lr)
        total.backward(g)
        assert torch.equal(lx.grad, g) and torch.equal(lr.grad, g) and (lw.grad is None or torch.all(lw.grad == 0))
    frozen = A.rms_norm(x, lw)  # the weight alone
    lw.grad = None
    frozen.backward(g)
    assert lw.grad is not None


def test_another_stream_and_graph():
    N, d = 300, 1024
    x, r, w, dy = rand(N, d, seed=27), rand(N, d, seed=28), rand(d, seed=29), rand(N, d, seed=30)
    ref = L.rms_norm(x, w, r)
    rb = L.rms_norm_bwd(ref["sum"], w, ref["rstd"], dy)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    o = L.rms_norm(x, w, r, stream=s)
    b = L.rms_norm_bwd(o["sum"], w, o["rstd"], dy, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(o["y"], ref["y"]) and torch.equal(b["dx"], rb["dx"]) and torch.equal(b["dweight"], rb["dweight"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o = L.rms_norm(x, w, r)
        b = L.rms_norm_bwd(o["sum"], w, o["rstd"], dy)
    x.copy_(rand(N, d, seed=31))
    for _ in range(2):
        g.replay()
    ref = L.rms_norm(x, w, r)
    rb = L.rms_norm_bwd(ref["sum"], w, ref["rstd"], dy)
    assert torch.equal(o["y"], ref["y"]) and torch.equal(b["dx"], rb["dx"]) and torch.equal(b["dweight"], rb["dweight"])


def test_two_backward_passes_at_once():
    """Each with its own workspace; and in a workspace of any content."""
    N, d = 700, 1344
    g = torch.Generator(device="cuda").manual_seed(31)
    x, dy = (torch.randn(2, N, d, device="cuda", generator=g).bfloat16() for _ in range(2))
    w = torch.rand(d, device="cuda", generator=g).bfloat16()
    f = [L.rms_norm(x[i], w) for i in range(2)]
    ref = [L.rms_norm_bwd(f[i]["sum"], w, f[i]["rstd"], dy[i]) for i in range(2)]
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [L.rms_norm_bwd(f[i]["sum"], w, f[i]["rstd"], dy[i], stream=s[i]) for i in range(2)]
        torch.cuda.synchronize()
        for a, b in zip(got, ref):
            assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dweight"], b["dweight"])
    ws = torch.full((L.lmh_workspace_size(L.make_shape(N, d, 1), L.ENTRY_RMS_NORM_BWD),), 255, dtype=torch.uint8, device="cuda")
    got = L.rms_norm_bwd(f[0]["sum"], w, f[0]["rstd"], dy[0], ws=ws)
    assert torch.equal(got["dx"], ref[0]["dx"]) and torch.equal(got["dweight"], ref[0]["dweight"])


def test_gradients_against_differences():
    """The formula's gradient, which the kernels are tested against, against central differences of
    the oracle's forward pass in fp64 (steps of 1e-5: both errors, of the step and of rounding,
    are below 1e-8 of values of order one)."""
    rng = np.random.default_rng(3)
    N, d, eps = 3, 64, 1e-6
    r, w, dy = rng.standard_normal((N, d)), rng.standard_normal(d), rng.standard_normal((N, d))

    def loss(r, w):
        return float((w * r / np.sqrt((r * r).mean(1, keepdims=True) + eps) * dy).sum())
    rstd = 1 / np.sqrt((r * r).mean(1, keepdims=True) + eps)
    n = r * rstd
    dx = rstd * (w * dy - n * (w * dy * n).mean(1, keepdims=True))
    dw = (dy * n).sum(0)
    h = 1e-5
    for j in (0, 17, 63):
        e = np.zeros(d)
        e[j] = h
        assert abs((loss(r, w + e) - loss(r, w - e)) / (2 * h) - dw[j]) < 1e-7
        for i in range(N):
            m = np.zeros((N, d))
            m[i, j] = h
            assert abs((loss(r + m, w) - loss(r - m, w)) / (2 * h) - dx[i, j]) < 1e-7
    # and the kernels' own, from bf16 inputs
    b = lambda a: torch.tensor(a, device="cuda").bfloat16()
    R, Wt, DY = b(r), b(w), b(dy)
    f = L.rms_norm(R, Wt, eps=eps)
    got = L.rms_norm_bwd(f["sum"], Wt, f["rstd"], DY)
    r, w, dy = (t.double().cpu().numpy() for t in (R, Wt, DY))
    num = np.zeros(d)
    for j in range(d):
        e = np.zeros(d)
        e[j] = h
        num[j] = (loss(r, w + e) - loss(r, w - e)) / (2 * h)
    err = np.abs(got["dweight"].double().cpu().numpy() - num)
    # one rounding to bf16 (2^-8), fp32 sums of three products, the differences' own 1e-7
    assert np.all(err <= 2.0 ** -8 * np.abs(num) + 1e-5 * np.abs(dy * r).sum(0) + 1e-7)


def test_one_tensor_as_x_and_residual():
    """The same tensor twice; and two leaves' gradients are not one tensor."""
    N, d = 33, 320
    x, w, g = rand(N, d, seed=32), rand(d, seed=33), rand(N, d, seed=34)
    f = L.rms_norm(x, w, x)
    b = L.rms_norm_bwd(f["sum"], w, f["rstd"], g)
    assert torch.equal(f["sum"], x + x)
    lx = x.clone().requires_grad_()
    A.rms_norm(lx, w, lx)[0].backward(g)
    assert torch.equal(lx.grad, b["dx"] + b["dx"])
    l1, l2 = x.clone().requires_grad_(), x.clone().requires_grad_()
    A.rms_norm(l1, w, l2)[0].backward(g)
    l1.grad.mul_(2)
    assert torch.equal(l2.grad, b["dx"]) and torch.equal(l1.grad, 2 * b["dx"])


def test_inputs_that_are_views():
    """Rows inside a larger buffer: contiguous, aligned to 16 bytes and no more."""
    N, d = 37, 192
    flat = [rand(1, N * d + 8, seed=35 + i).flatten() for i in range(3)]
    x, r, dy = (t[8:].view(N, d) for t in flat)
    w = rand(1, d + 8, seed=40).flatten()[8:]
    f, ref = L.rms_norm(x, w, r), L.rms_norm(x.clone(), w.clone(), r.clone())
    b, rb = (L.rms_norm_bwd(o["sum"], w, o["rstd"], dy) for o in (f, ref))
    q, rq = L.rms_norm(x, w, r, fp8=True), L.rms_norm(x.clone(), w.clone(), r.clone(), fp8=True)
    assert torch.equal(f["y"], ref["y"]) and torch.equal(b["dx"], rb["dx"]) and torch.equal(b["dweight"], rb["dweight"])
    assert torch.equal(q["q"].view(torch.uint8), rq["q"].view(torch.uint8)) and torch.equal(q["scale"], rq["scale"])


def test_backward_of_rows_far_from_one():
    """Rows so large that the forward gives 0 (rstd = 0): dx = dsum there and no share of dweight.
    And small rows with small gradients, whose products r dy would be subnormal."""
    N, d = 6, 192
    x, w, dy, ds = rand(N, d, seed=41), rand(d, seed=42), rand(N, d, seed=43, scale=30), rand(N, d, seed=44)
    x[2], x[4] = 3e38, -2e38
    f = L.rms_norm(x, w)
    assert torch.all(f["rstd"][[2, 4]] == 0) and torch.all(f["y"][[2, 4]] == 0)
    b = L.rms_norm_bwd(f["sum"], w, f["rstd"], dy, ds)
    assert torch.equal(b["dx"][[2, 4]], ds[[2, 4]])
    rest = [0, 1, 3, 5]
    part = L.rms_norm_bwd(f["sum"][rest].clone(), w, f["rstd"][rest].clone(), dy[rest].clone(), ds[rest].clone())
    assert torch.equal(b["dx"][rest], part["dx"])
    r, wf, g = f64(x[rest]), f64(w), f64(dy[rest])
    _, dw = S.rms_norm_bwd(r, wf, 1e-6, g)
    n = r / np.sqrt((r * r).mean(1, keepdims=True) + 1e-6)
    assert np.all(np.abs(f64(b["dweight"]) - dw) <= BF * np.abs(dw) + 2 * E32 * (np.abs(g * n)).sum(0))

    x, dy = rand(N, d, seed=45, scale=1e-15), rand(N, d, seed=46, scale=1e-27)
    f = L.rms_norm(x, w, eps=0.0)
    b = L.rms_norm_bwd(f["sum"], w, f["rstd"], dy)
    r, g = f64(x), f64(dy)
    dx, dw = S.rms_norm_bwd(r, wf, 0.0, g)
    rstd = 1 / np.sqrt((r * r).mean(1, keepdims=True))
    n = np.abs(r * rstd)
    terms = rstd * (np.abs(wf * g) + n * (np.abs(wf * g) * n).mean(1, keepdims=True))
    assert np.all(np.abs(f64(b["dx"]) - dx) <= BF * np.abs(dx) + 3 * E32 * terms)
    assert np.all(np.abs(f64(b["dweight"]) - dw) <= BF * np.abs(dw) + 2 * E32 * (np.abs(g) * n).sum(0))


@pytest.mark.parametrize("both", [False, True])
def test_autograd_of_gradients_at_any_address(both):
    """An upstream gradient is wherever torch has it: here one element behind an aligned address."""
    N, d = 5, 128
    x, r, w = rand(N, d, seed=47), rand(N, d, seed=48), rand(d, seed=49)
    first = torch.zeros(1, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    lx, lr, lw = (t.clone().requires_grad_() for t in (x, r, w))
    H, total = A.rms_norm(lx, lw, lr)
    parts = [first, H.flatten()] + ([total.flatten()] if both else [])
    g = rand(1, 1 + (len(parts) - 1) * N * d, seed=50).flatten()
    torch.cat(parts).backward(g)
    f = L.rms_norm(x, w, r)
    dy = g[1:1 + N * d].clone().view(N, d)
    b = L.rms_norm_bwd(f["sum"], w, f["rstd"], dy, g[1 + N * d:].clone().view(N, d) if both else None)
    assert torch.equal(lx.grad, b["dx"]) and torch.equal(lr.grad, b["dx"]) and torch.equal(lw.grad, b["dweight"])
