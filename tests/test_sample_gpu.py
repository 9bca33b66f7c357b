"""Sampling against the fp64 oracle: tokens have to be equal. The kernel's weights are off by less
than 2^-40 of the row's largest, so with random u a token differs from the oracle's with a
probability of at most V * 2^-39 per row (each token's interval moves by less than that), below 1e-6
for every row here. The log-prob is rounded to fp32 once (2^-24), and the sum of weights in it is
formed of fp32 exponentials 2^y, y = log2(e) (z - zmax) / tau: 2^-22 of each for the exponential,
three roundings of y, 3 * 2^-24 |y| ln2, and 2^-41 for its rounding to a whole number. Relative to
the sum that is 2^-22 + 3 * 2^-24 E[|z - zmax| / tau] + V * 2^-41, the expectation over the row's
softmax, as log2(e) ln2 = 1."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import lm_head_cross_tcgen05_b200 as L
from oracle import serving_oracle as S

pytestmark = pytest.mark.gpu

f32 = torch.float32


def f64(t):
    return t.detach().cpu().double().numpy()


def logits(N, V, seed, scale=3.0, dtype=f32, digits=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.randn(N, V, device="cuda", generator=g) * scale
    if digits is not None:
        z = (z * 10 ** digits).round() / 10 ** digits
    return z.to(dtype), torch.rand(N, device="cuda", generator=g)


def check(z, u, tau=None, k=None, p=None, m=None, flags=0):
    o = L.sample(z, u, temperature=tau, top_k=k, top_p=p, min_p=m)
    assert L.lmh_read_errors(o["workspace"]) == flags
    N = z.shape[0]

    def row(v, i, off, t):
        if v is None:
            return off
        return float(v[i]) if isinstance(v, torch.Tensor) else float(torch.tensor(v, dtype=t))
    zz, uu, got, lp = f64(z), f64(u), o["tokens"].tolist(), f64(o["logprob"])
    for i in range(N):
        tau_i = row(tau, i, 1.0, f32) or 1.0
        want, wlp = S.sample(zz[i], uu[i], tau_i, int(row(k, i, 0, torch.int64)), row(p, i, 1.0, f32), row(m, i, 0.0, f32))
        assert got[i] == want, (i, got[i], want)
        if want >= 0:
            t0 = (zz[i] - zz[i].max()) / tau_i
            e = np.exp(t0)
            away = -(e[e > 0] * t0[e > 0]).sum() / e.sum()
            assert abs(lp[i] - wlp) <= 2.0 ** -24 * (abs(wlp) + 1) + 2.0 ** -22 + 3 * 2.0 ** -24 * away + len(t0) * 2.0 ** -41
        else:
            assert lp[i] == 0
    return o


FILTERS = [dict(), dict(k=1), dict(k=50), dict(p=0.9), dict(p=0.3), dict(m=0.05), dict(k=40, p=0.8), dict(k=2000, p=0.95, m=0.001),
           dict(tau=0.6), dict(tau=1.7, k=100, p=0.99), dict(tau=0.05, p=0.5, m=0.1), dict(p=0.0), dict(k=-3, p=1.5, m=-1.0), dict(m=2.0)]


@pytest.mark.parametrize("kw", FILTERS)
@pytest.mark.parametrize("V", [1, 2, 31, 513, 5000, 32000, 100003])
def test_scalars(V, kw):
    check(*logits(6 if V < 100000 else 3, V, seed=V), **kw)


@pytest.mark.parametrize("kw", FILTERS)
@pytest.mark.parametrize("dtype,digits", [(torch.bfloat16, None), (f32, 1)])
def test_equal_logits_at_the_borders(dtype, digits, kw):
    check(*logits(8, 9001, seed=7, dtype=dtype, digits=digits), **kw)


@pytest.mark.parametrize("kw", [dict(), dict(k=1), dict(k=700), dict(k=30000), dict(p=0.5), dict(p=0.9, k=20000), dict(m=1.0), dict(p=0.001)])
@pytest.mark.parametrize("V", [3000, 65536, 150001])
def test_all_logits_equal(V, kw):
    z, u = logits(3, V, seed=8)
    check(torch.full_like(z, -1.25), u, **kw)


@pytest.mark.parametrize("kw", [dict(k=3000), dict(p=0.7), dict(k=9000, p=0.9), dict(k=5)])
def test_crowded_buckets(kw):
    """One linear bucket holds most of the row: it is split by the bits of the keys."""
    g = torch.Generator(device="cuda").manual_seed(9)
    z = 5 + 1e-5 * torch.randn(4, 40000, device="cuda", generator=g)
    z[1] = (z[1] - 5) * 1e-30  # around zero, both signs
    z[2, ::2] = 5
    z[3] = torch.where(z[3] > 5, 0.0, -0.0)  # equal zeros of both signs
    z[0, 17] = 9
    check(z, torch.rand(4, device="cuda", generator=g), **kw)


def test_one_bucket_of_ties_and_neighbours():
    z, u = logits(2, 30000, seed=10, scale=1e-6)
    z[:, 5000:] = z[:, 5000:].round(decimals=6)
    for kw in (dict(k=2), dict(k=4999), dict(k=15000), dict(p=0.4)):
        check(z, u, **kw)


@pytest.mark.parametrize("dtype", [f32, torch.bfloat16])
def test_per_row_parameters(dtype):
    N, V = 64, 20011
    z, u = logits(N, V, seed=11, dtype=dtype)
    g = torch.Generator(device="cuda").manual_seed(12)

    def pick(v, t):
        return torch.tensor(v, device="cuda", dtype=t)[torch.randint(len(v), (N,), device="cuda", generator=g)]
    check(z, u, tau=pick([0.3, 0.8, 1.0, 2.5], f32), k=pick([0, 1, 7, 50, 900, V, V + 5, -1], torch.int32),
          p=pick([0.0, 0.2, 0.9, 0.999, 1.0], f32), m=pick([0.0, 0.01, 0.3, 1.0], f32))


def test_scalar_times_row_temperature():
    z, u = logits(5, 777, seed=13)
    row = torch.tensor([0.5, 1.0, 2.0, 0.7, 3.0], device="cuda")
    shape = L.make_shape(5, 64, 777, temperature=row)
    shape.temperature = 0.5
    tok, lp = torch.empty(5, dtype=torch.int32, device="cuda"), torch.empty(5, device="cuda")
    ws = L.workspace(shape, L.ENTRY_SAMPLE, "cuda")
    L.lmh_sample(shape, L.make_sampling(5, top_k=9), z, u, tok, lp, workspace=ws)
    ref = L.sample(z, u, temperature=row * 0.5, top_k=9)
    assert torch.equal(tok, ref["tokens"]) and torch.equal(lp, ref["logprob"])


@pytest.mark.parametrize("dtype", [f32, torch.bfloat16])
def test_masked_rows(dtype):
    N, V = 12, 6007
    z, u = logits(N, V, seed=14, dtype=dtype)
    low = torch.finfo(dtype).min
    z[0, 1:] = -torch.inf          # one left
    z[1] = -torch.inf              # none left
    z[2, :5000] = low              # the type's lowest value
    z[3] = low                     # all at the lowest value
    z[4, 7] = float("nan")
    z[5, 6000] = torch.inf
    z[6, 100:] = -torch.inf
    z[7, :] = low
    z[7, 33] = -low                # the whole range of the type
    z[8] = -torch.inf
    z[8, -1] = low
    z[9, 3] = -low
    for kw in (dict(), dict(k=50), dict(p=0.9), dict(k=20, p=0.5, m=0.1), dict(tau=0.01, p=0.99), dict(tau=1e30, p=0.5), dict(tau=1e38), dict(tau=1e38, p=0.9, k=300), dict(m=0.5)):
        o = check(z, u, flags=L.DEVERR_NONFINITE, **kw)
        assert o["tokens"][[1, 4, 5]].tolist() == [-1] * 3 and torch.all(o["logprob"][[1, 4, 5]] == 0)


def test_extreme_temperatures():
    z, u = logits(4, 3000, seed=15)
    for tau in (1e-38, 1e-20, 1e-3, 1e3, 1e20, 1e38):
        for kw in (dict(), dict(k=10), dict(p=0.5), dict(m=0.2)):
            check(z, u, tau=tau, **kw)


def test_parameters_out_of_range_are_flagged():
    z, u = logits(8, 500, seed=16)
    nan = float("nan")
    u[0], u[1], u[2], u[3] = 1.0, -0.5, nan, float("inf")
    p = torch.tensor([0.9] * 6 + [nan, 0.9], device="cuda")
    o = L.sample(z, u, top_p=p)
    assert L.lmh_read_errors(o["workspace"]) == L.DEVERR_SAMPLING
    ok_u = u.clone()
    ok_u[0] = ok_u[3] = 1 - 2.0 ** -24  # no kept token is so unlikely that this is not the last one
    ok_u[1] = ok_u[2] = 0
    p[6] = 1.0
    assert torch.equal(o["tokens"], check(z, ok_u, p=p)["tokens"])
    tau = torch.tensor([1.0, 0.0, -1.0, nan, float("inf"), 2.0, 1.0, 1.0], device="cuda")
    o = L.sample(z, ok_u, temperature=tau)
    assert L.lmh_read_errors(o["workspace"]) == L.DEVERR_TEMPERATURE
    tau[1:5] = 1
    assert torch.equal(o["tokens"], check(z, ok_u, tau=tau)["tokens"])


@pytest.mark.parametrize("V,dtype", [(262144, f32), (450001, f32), (450001, torch.bfloat16), (1000003, f32)])
def test_long_rows(V, dtype):
    """Up to and past what a cluster's shared memory holds."""
    z, u = logits(2, V, seed=17, dtype=dtype)
    for kw in (dict(), dict(k=50, p=0.9), dict(p=0.97), dict(k=60000)):
        check(z, u, **kw)


def test_many_rows_and_each_alone():
    N, V = 700, 4099
    z, u = logits(N, V, seed=18)
    o = check(z, u, k=30, p=0.9, tau=0.8)
    for i in (0, 1, 350, 699):
        one = L.sample(z[i:i + 1].clone(), u[i:i + 1].clone(), top_k=30, top_p=0.9, temperature=0.8)
        assert torch.equal(one["tokens"], o["tokens"][i:i + 1]) and torch.equal(one["logprob"], o["logprob"][i:i + 1])


def test_offsets_past_32_bits():
    N, V = 4200, 524288
    z = torch.zeros(N, V, device="cuda", dtype=torch.bfloat16)
    zz, u = logits(3, V, seed=19, dtype=torch.bfloat16)
    z[-3:] = zz
    uu = torch.zeros(N, device="cuda")
    uu[-3:] = u
    o = L.sample(z, uu, top_k=50)
    ref = check(zz, u, k=50)
    assert torch.equal(o["tokens"][-3:], ref["tokens"]) and torch.all(o["tokens"][:-3] == 0)


def test_u_covers_every_token_by_its_weight():
    """Equal weights, u on and beside every border."""
    V = 64
    u = torch.arange(0, V * 4, device="cuda", dtype=f32) / (V * 4)
    z = torch.zeros(V * 4, V, device="cuda")
    z[:, 10:20] = -torch.inf
    kept = [i for i in range(V) if not 10 <= i < 20]
    want = [kept[int(x * len(kept))] for x in u.double().tolist()]
    assert L.sample(z, u)["tokens"].tolist() == want


def test_logprob_is_that_of_the_head():
    """sample()'s log-prob is lmh_logprob's for the same token, up to the logits' own rounding."""
    N, V, d = 40, 1500, 128
    g = torch.Generator(device="cuda").manual_seed(20)
    H, W = torch.randn(N, d, device="cuda", generator=g).bfloat16(), (0.1 * torch.randn(V, d, device="cuda", generator=g)).bfloat16()
    z = H.double() @ W.double().t()
    o = L.sample(z.float(), torch.rand(N, device="cuda", generator=g), temperature=0.7, top_p=0.9)
    lp = L.logprob(H, W, o["tokens"], temperature=0.7)["logprob"]
    assert float((lp - o["logprob"]).abs().max()) < 2e-3


def test_no_rows():
    o = L.sample(torch.empty(0, 50, device="cuda"), torch.empty(0, device="cuda"))
    assert o["tokens"].shape == (0,)


def test_another_stream_and_two_graphs():
    z, u = logits(20, 30011, seed=21)
    kw = dict(top_k=50, top_p=0.9)
    ref = L.sample(z, u, **kw)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    o = L.sample(z, u, stream=s, **kw)
    s.synchronize()
    assert torch.equal(o["tokens"], ref["tokens"])
    outs, graphs = [], []
    for kw in (dict(top_k=50), dict(top_p=0.9)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(L.sample(z, u, **kw))
        graphs.append(g)
    z2, u2 = logits(20, 30011, seed=22)
    z.copy_(z2), u.copy_(u2)
    torch.cuda.synchronize()
    for g, st in zip(graphs, (s, torch.cuda.Stream())):
        with torch.cuda.stream(st):
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0]["tokens"], check(z, u, k=50)["tokens"])
    assert torch.equal(outs[1]["tokens"], check(z, u, p=0.9)["tokens"])


def test_decode_step():
    """norm -> 8-bit logits -> token, with scores for the drawn tokens from the same logits."""
    N, V, d = 9, 3001, 320
    g = torch.Generator(device="cuda").manual_seed(23)
    x, r = torch.randn(N, d, device="cuda", generator=g).bfloat16(), torch.randn(N, d, device="cuda", generator=g).bfloat16()
    w = torch.rand(d, device="cuda", generator=g).bfloat16()
    W = (0.1 * torch.randn(V, d, device="cuda", generator=g)).bfloat16()
    u = torch.rand(N, device="cuda", generator=g)
    W8, ws = L.quantize_fp8(W)
    o = L.next_tokens(x, w, W8, ws, u, r, temperature=0.9, top_k=30, top_p=0.95)
    n = L.rms_norm(x, w, r, fp8=True)
    z = L.fp8_logits(n["q"], n["scale"], W8, ws)["logits"]
    assert torch.equal(o["logits"], z)
    ref = check(z, u, tau=0.9, k=30, p=0.95)
    assert torch.equal(o["tokens"], ref["tokens"]) and torch.equal(o["logprob"], ref["logprob"])
    # the 8-bit head is the bf16 head up to the two quantisations
    y = L.rms_norm(x, w, r)["y"]
    zb = y.double() @ W.double().t()
    mags = y.double().abs() @ W.double().abs().t()
    assert torch.all((z.double() - zb).abs() <= (2 * 2.0 ** -4 + 2.0 ** -7) * mags)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = L.next_tokens(x, w, W8, ws, u, r, temperature=0.9, top_k=30, top_p=0.95)
    x.copy_(x.flip(0)), r.copy_(r.flip(0)), u.copy_(u.flip(0))
    graph.replay()
    assert torch.equal(c["tokens"], o["tokens"].flip(0))


@pytest.mark.parametrize("scale", [0.5, 1.5, 4.0])
@pytest.mark.parametrize("V", [40009, 140000])
def test_long_prefixes(V, scale):
    """Flat rows, whose prefixes hold from a few to most of the logits."""
    z, u = logits(2, V, seed=24, scale=scale)
    for kw in (dict(p=0.05), dict(p=0.5), dict(p=0.9), dict(p=0.995), dict(p=0.9, m=1e-4), dict(p=0.7, m=0.3), dict(k=5000, p=0.9),
               dict(k=30000, p=0.5, m=1e-3), dict(k=V - 1, p=0.999)):
        check(z, u, **kw)


@pytest.mark.parametrize("kw", [dict(k=600), dict(k=900, p=0.97), dict(p=0.8), dict(k=200, p=0.5)])
def test_likely_tokens_in_one_run_of_ids(kw):
    z, u = logits(3, 150001, seed=25, scale=0.5)
    z[0, 40000:41000] += 30
    z[1, :1000] += 30
    z[2, -1000:] += 30
    check(z, u, **kw)


@pytest.mark.parametrize("kw", [dict(p=0.9), dict(k=130), dict(k=400, p=0.6), dict(k=900), dict(m=0.02)])
@pytest.mark.parametrize("V", [400, 1900])
def test_few_different_values(V, kw):
    check(*logits(4, V, seed=26, scale=1.0, digits=0), **kw)


@pytest.mark.parametrize("kw", [dict(), dict(k=20), dict(p=0.9), dict(k=3000)])
def test_workspace_of_any_content(kw):
    z, u = logits(5, 33001, seed=27)
    names = dict(k="top_k", p="top_p")
    kw2 = {names[k]: v for k, v in kw.items()}
    ref = check(z, u, **kw)
    for fill in (0, 255):
        ws = torch.full_like(ref["workspace"], fill)
        o = L.sample(z, u, ws=ws, **kw2)
        assert torch.equal(o["tokens"], ref["tokens"]) and L.lmh_read_errors(ws) == 0
    # left by a call of other sizes
    small = L.sample(z[:2, :1000].contiguous(), u[:2], ws=ws, **kw2)
    assert torch.equal(small["tokens"], check(z[:2, :1000].contiguous(), u[:2], **kw)["tokens"])


def test_two_calls_at_once():
    z, u = logits(30, 70001, seed=28)
    ref = [L.sample(z, u, top_p=0.9), L.sample(z, u, top_k=3000)]
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        o = [L.sample(z, u, top_p=0.9, stream=s[0]), L.sample(z, u, top_k=3000, stream=s[1])]
        torch.cuda.synchronize()
        for a, b in zip(o, ref):
            assert torch.equal(a["tokens"], b["tokens"]) and torch.equal(a["logprob"], b["logprob"])


@pytest.mark.parametrize("dtype", [f32, torch.bfloat16])
@pytest.mark.parametrize("by", [1, 3, 5])
def test_logits_at_any_address(dtype, by):
    """Aligned to their element only; u, tokens and parameters to theirs."""
    z, u = logits(4, 40000, seed=29, dtype=dtype)
    flat = torch.full((z.numel() + by + 7,), 50.0, device="cuda", dtype=dtype)  # what lies beside is never read as a logit
    flat[by:by + z.numel()].copy_(z.flatten())
    moved = flat[by:by + z.numel()].view(z.shape)
    uu = torch.zeros(5, device="cuda")
    uu[1:].copy_(u)
    for kw in (dict(), dict(k=40), dict(p=0.9), dict(k=4000, p=0.8)):
        ref = check(z, u, **kw)
        o = check(moved, uu[1:], **kw)
        assert torch.equal(o["tokens"], ref["tokens"]) and torch.equal(o["logprob"], ref["logprob"])


def below(V, bits, dtype):
    """A logit of the type that is next to `bits` above or below 2^-F of a largest one of 0; F as in lmh.h."""
    F = min(50, 62 - int(np.ceil(np.log2(V))))
    return F, float(torch.tensor(-(F - bits) * np.log(2.0)).to(dtype))


ALL_FILTERS = [dict(), dict(k=50), dict(k=2000), dict(p=0.9), dict(m=1e-30), dict(m=0.05), dict(k=40, p=0.8), dict(k=1500, p=0.9, m=1e-30)]


@pytest.mark.parametrize("kw", ALL_FILTERS)
@pytest.mark.parametrize("dtype", [f32, torch.bfloat16])
@pytest.mark.parametrize("V", [768, 5000, 151936])
def test_blocks_of_weightless_logits_are_passed_over(V, dtype, kw):
    """256 logits, each too small to be drawn though all of them together are not: u at their place."""
    F, low = below(V, -1.45, dtype)
    e = np.exp(low)
    assert e < 2.0 ** -(F + 1) and 250 * e > 2.0 ** -F
    z = torch.full((5, V), -torch.inf, device="cuda")
    z[0, 1:256], z[0, 256:] = low, 0.0           # id 0 masked, and the first block weightless
    z[1, :256], z[1, 256:] = low, 0.0
    z[2, 256:512], z[2, 600:] = low, 0.0         # nothing, a weightless block, then the rest
    z[3, 7], z[3, 256:512], z[3, 700] = 0.0, low, 0.0
    z[4, 7], z[4, 512:768], z[4, 300] = 0.0, low, 0.0  # behind the last that can be drawn
    u = torch.tensor([0.0, 0.0, 0.0, 0.5, 1 - 2.0 ** -24], device="cuda")
    z = z.to(dtype)
    names = dict(k="top_k", p="top_p", m="min_p")
    o = L.sample(z, u, **{names[a]: v for a, v in kw.items()})
    # with k = 40 of equal ones p = 0.8 keeps 32, which start with the first; u = 0.5 halves two
    want = [256, 256, 600, 700, 300]
    assert L.lmh_read_errors(o["workspace"]) == 0 and o["tokens"].tolist() == want
    lp = -np.log(np.exp(f64(z)).sum(1))
    assert np.all(np.abs(f64(o["logprob"]) - lp) <= 2.0 ** -24 * (np.abs(lp) + 1) + 2.0 ** -22)


@pytest.mark.parametrize("kw", ALL_FILTERS)
@pytest.mark.parametrize("dtype", [f32, torch.bfloat16])
@pytest.mark.parametrize("V", [768, 5000, 151936])
def test_the_least_probability_that_is_drawn(V, dtype, kw):
    """At u = 0 the first id whose probability is at least 2^-F of the largest is drawn."""
    F, under = below(V, -0.5, dtype)
    _, over = below(V, 0.25, dtype)
    assert np.exp(under) < 2.0 ** -(F + 0.25) and np.exp(over) > 2.0 ** -F
    z = torch.full((3, V), -torch.inf, device="cuda")
    z[0, 0], z[0, 300] = under, 0.0
    z[1, :256], z[1, 300] = under, 0.0
    z[2, 0], z[2, 5], z[2, 300] = under, over, 0.0
    names = dict(k="top_k", p="top_p", m="min_p")
    o = L.sample(z.to(dtype), torch.zeros(3, device="cuda"), **{names[a]: v for a, v in kw.items()})
    far = 300 if kw.get("p") or kw.get("m") == 0.05 else 5  # top-p and min-p leave the largest alone
    assert o["tokens"].tolist() == [300, 300, far]


@pytest.mark.parametrize("kw", [dict(m=1.0), dict(m=2.0), dict(m=0.5), dict(k=3000, m=1.0), dict(p=0.9, m=1.0), dict(p=0.5), dict()])
@pytest.mark.parametrize("V", [300, 40000])
@pytest.mark.parametrize("dtype", [f32, torch.bfloat16])
def test_zeros_of_both_signs_are_equal(dtype, V, kw):
    z, u = logits(8, V, seed=30)
    z = torch.where(z > 2, 0.0, torch.where(z > 0, -0.0, -z.abs()))
    for tau in (None, 1e-38):
        check(z.to(dtype), u, tau=tau, **kw)


@pytest.mark.parametrize("kw", [dict(), dict(p=0.6)])
@pytest.mark.parametrize("V", [300, 40000])
def test_subnormal_logits_at_tiny_temperatures(V, kw):
    z, u = logits(4, V, seed=31, scale=4e-39)
    check(z, u, tau=2e-39, **kw)
    check(z, u, tau=1.5e-38, **kw)


def test_parameters_of_rows_without_a_sum_are_flagged():
    z, u = logits(3, 500, seed=32)
    z[1] = -torch.inf
    nan = float("nan")
    good = torch.full((3,), 0.9, device="cuda")
    bad = good.clone()
    bad[1] = nan
    for kw in (dict(u=u), dict(u=u, top_p=good)):
        o = L.sample(z, **kw)
        assert L.lmh_read_errors(o["workspace"]) == L.DEVERR_NONFINITE
    for kw, flag in ((dict(top_p=bad), L.DEVERR_SAMPLING), (dict(min_p=bad), L.DEVERR_SAMPLING), (dict(temperature=bad), L.DEVERR_TEMPERATURE)):
        o = L.sample(z, u, **kw)
        assert L.lmh_read_errors(o["workspace"]) == L.DEVERR_NONFINITE | flag
        assert o["tokens"][1] == -1 and o["logprob"][1] == 0
    u[1] = 1.5
    assert L.lmh_read_errors(L.sample(z, u)["workspace"]) == L.DEVERR_NONFINITE | L.DEVERR_SAMPLING


@pytest.mark.parametrize("scalar,row", [(1e-44, 2.9e38), (2.9e38, 1e-38)])
def test_product_of_far_apart_temperatures(scalar, row):
    """Only their product counts, and it is an ordinary number."""
    N, V = 5, 3000
    scalar, row = float(np.float32(scalar)), float(np.float32(row))
    z, u = logits(N, V, seed=33, scale=3 * scalar * row)
    rows = torch.full((N,), row, device="cuda")
    shape = L.make_shape(N, 64, V, temperature=rows)
    shape.temperature = scalar
    for kw in (dict(), dict(top_k=9), dict(min_p=0.01), dict(top_p=0.5)):
        tok, lp = torch.empty(N, dtype=torch.int32, device="cuda"), torch.empty(N, device="cuda")
        ws = L.workspace(shape, L.ENTRY_SAMPLE, "cuda")
        L.lmh_sample(shape, L.make_sampling(N, **kw), z, u, tok, lp, workspace=ws)
        exact = {a: v if a == "top_k" else float(np.float32(v)) for a, v in kw.items()}
        zz, uu, tau = f64(z), f64(u), scalar * row
        for i in range(N):
            t, w = S.sample(zz[i], uu[i], tau, **exact)
            t0 = (zz[i] - zz[i].max()) / tau
            away = -(np.exp(t0) * t0).sum() / np.exp(t0).sum()
            # as in check(); y has one rounding more, that of the product
            assert tok[i] == t and abs(float(lp[i]) - w) <= 2.0 ** -24 * (abs(w) + 1) + 2.0 ** -22 + 4 * 2.0 ** -24 * away + V * 2.0 ** -41


@pytest.mark.parametrize("scalar,row,scale", [(1.0, 1e-40, 2e-40), (1.0, 5e-39, 1e-38), (1e-20, 1e-22, 1e-42), (1e19, 1e20, 1e38), (1e38, 2.9e38, 1e38)])
@pytest.mark.parametrize("kw", [dict(), dict(top_k=300), dict(min_p=0.01), dict(top_p=0.5)])
def test_logprob_at_temperatures_whose_inverse_is_no_normal_number(scalar, row, scale, kw):
    N, V = 4, 2500
    z, u = logits(N, V, seed=34, scale=1.0)
    z = z.clamp(-3, 3) * scale
    z[0, ::2] = -3 * scale
    rows = torch.full((N,), row, device="cuda")
    shape = L.make_shape(N, 64, V, temperature=rows)
    shape.temperature = scalar
    tok, lp = torch.empty(N, dtype=torch.int32, device="cuda"), torch.empty(N, device="cuda")
    ws = L.workspace(shape, L.ENTRY_SAMPLE, "cuda")
    L.lmh_sample(shape, L.make_sampling(N, **kw), z, u, tok, lp, workspace=ws)
    assert L.lmh_read_errors(ws) == 0
    exact = {a: v if a == "top_k" else float(np.float32(v)) for a, v in kw.items()}
    zz, uu, tau = f64(z), f64(u), float(np.float32(scalar)) * float(rows[0])
    for i in range(N):
        t, w = S.sample(zz[i], uu[i], tau, **exact)
        # the sum is in fp64 here: the log-prob has its own rounding alone
        assert tok[i] == t and abs(float(lp[i]) - w) <= 2.0 ** -24 * (abs(w) + 1) + V * 2.0 ** -41
