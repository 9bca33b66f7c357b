"""Pins of the serving oracle: differences, closed forms and brute force on tiny inputs (CPU)."""
import math

import numpy as np
import pytest

from oracle import serving_oracle as S


def test_norm_gradients_are_the_differences():
    rng = np.random.default_rng(0)
    r, w, dy, ds = rng.normal(size=(3, 8)), rng.normal(size=8), rng.normal(size=(3, 8)), rng.normal(size=(3, 8))
    eps, h = 1e-3, 1e-6

    def loss(r, w):
        return (S.rms_norm(r, w, eps)[0] * dy).sum() + (r * ds).sum()
    dx, dw = S.rms_norm_bwd(r, w, eps, dy, ds)
    for idx in np.ndindex(r.shape):
        e = np.zeros_like(r)
        e[idx] = h
        assert (loss(r + e, w) - loss(r - e, w)) / (2 * h) == pytest.approx(dx[idx], abs=1e-7)
    for j in range(8):
        e = np.zeros_like(w)
        e[j] = h
        assert (loss(r, w + e) - loss(r, w - e)) / (2 * h) == pytest.approx(dw[j], abs=1e-7)


def test_norm_of_a_constant_row():
    y, rstd = S.rms_norm(np.full((1, 4), -3.0), np.array([1.0, 2.0, 0.0, -1.0]), 0.0)
    assert np.allclose(y, [[-1, -2, 0, 1]]) and rstd[0] == pytest.approx(1 / 3)


def test_block_scales_by_loops():
    x = np.random.default_rng(1).normal(size=(130, 192))
    x[:, 128:][:128] = 0
    s = S.block_scales(x, 128)
    assert s.shape == (2, 2)
    assert s[0, 1] == 2.0 ** -100 / 448
    assert s[1, 0] == max(abs(x[i, j]) for i in (128, 129) for j in range(128)) / 448
    assert np.array_equal(S.block_scales(x, 1)[5], [np.abs(x[5, :128]).max() / 448, 2.0 ** -100 / 448])
    full = S.expand(s, 128, x.shape)
    assert full.shape == x.shape and full[129, 191] == s[1, 1] and full[127, 127] == s[0, 0]


def test_scaled_product_by_loops():
    rng = np.random.default_rng(2)
    h, w = rng.integers(-8, 9, (3, 192)).astype(float), rng.integers(-8, 9, (129, 192)).astype(float)
    hs, ws = rng.uniform(0.1, 1, (3, 2)), rng.uniform(0.1, 1, (2, 2))
    z = S.logits(h, hs, w, ws)
    for n, v in ((0, 0), (2, 127), (1, 128)):
        want = sum(h[n, k] * hs[n, k // 128] * w[v, k] * ws[v // 128, k // 128] for k in range(192))
        assert z[n, v] == pytest.approx(want, rel=1e-12)


def brute_kept(z, tau, k, p, m):
    """Takes ids one by one, the largest remaining logit (lowest id) first."""
    left, chosen = list(range(len(z))), []
    while left and (k <= 0 or len(chosen) < k):
        best = max(left, key=lambda i: (z[i], -i))
        chosen.append(best)
        left.remove(best)
    w = [math.exp((z[i] - z[chosen[0]]) / tau) for i in chosen]
    if p < 1:
        n = 1
        while n < len(w) and math.fsum(w[:n]) < p * math.fsum(w):
            n += 1
        chosen, w = chosen[:n], w[:n]
    return sorted(i for i, x in zip(chosen, w) if x >= m)


@pytest.mark.parametrize("seed", range(30))
def test_kept_by_brute_force(seed):
    rng = np.random.default_rng(seed)
    z = np.round(rng.normal(size=12) * 2, 1 if seed % 2 else 6)  # odd seeds hold equal logits
    tau, k, p, m = rng.choice([0.5, 1.0, 1.7]), int(rng.integers(0, 14)), rng.choice([0.0, 0.3, 0.9, 1.0]), rng.choice([0.0, 0.05, 0.3])
    got = S.kept(z, tau, k, p, m).tolist()
    assert got == brute_kept(z.tolist(), tau, k, p, m)
    ids = np.array(got)
    e = np.exp(z[ids] / tau)
    cuts = np.concatenate([[0], np.cumsum(e) / e.sum()])
    for j, i in enumerate(ids):  # the middle of a token's interval draws it
        assert S.sample(z, (cuts[j] + cuts[j + 1]) / 2, tau, k, p, m)[0] == i
    t, lp = S.sample(z, 0.0, tau, k, p, m)
    assert t == ids[0] and lp == pytest.approx(z[t] / tau - math.log(sum(math.exp(x / tau) for x in z)))


def test_rows_without_a_finite_log_sum_exp():
    for bad in ([-np.inf, -np.inf], [0, np.nan], [0, np.inf]):
        assert S.sample(np.array(bad), 0.5) == (-1, 0.0)
