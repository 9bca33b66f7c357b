"""fp64 definitions of the operators around the head: RMS norm with residual, its gradients, block
scales of 8-bit matrices, the scaled product, and sampling. Plain numpy, no code shared with the
GPU path."""
from __future__ import annotations

import math

import numpy as np

BLOCK = 128
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100


def rms_norm(r, w, eps):
    """r [N, d] is the stored (already rounded) sum. -> y, rstd"""
    r, w = np.asarray(r, np.float64), np.asarray(w, np.float64)
    rstd = 1.0 / np.sqrt((r * r).mean(axis=1) + eps)
    return w * r * rstd[:, None], rstd


def rms_norm_bwd(r, w, eps, dy, dsum=None):
    """-> dx, dweight of sum(dy * y) + sum(dsum * r)."""
    r, w, dy = (np.asarray(a, np.float64) for a in (r, w, dy))
    _, rstd = rms_norm(r, w, eps)
    n = r * rstd[:, None]
    c = (w * dy * n).mean(axis=1, keepdims=True)
    dx = (w * dy - n * c) * rstd[:, None]
    if dsum is not None:
        dx = dx + np.asarray(dsum, np.float64)
    return dx, (dy * n).sum(axis=0)


def block_scales(x, block_rows):
    """One scale per block of block_rows x 128 of x: max(amax, 2^-100) / 448."""
    x = np.abs(np.asarray(x, np.float64))
    rows, d = x.shape
    out = np.empty((-(-rows // block_rows), -(-d // BLOCK)))
    for i in range(out.shape[0]):
        for j in range(out.shape[1]):
            b = x[i * block_rows:(i + 1) * block_rows, j * BLOCK:(j + 1) * BLOCK]
            out[i, j] = np.maximum(b.max(), AMAX_FLOOR) / E4M3_MAX
    return out


def expand(scale, block_rows, shape):
    rows, d = shape
    return np.repeat(np.repeat(scale, block_rows, 0)[:rows], BLOCK, 1)[:, :d]


def logits(h8, h_scale, w8, w_scale):
    """h8 [N, d], w8 [V, d]: the e4m3 values as numbers."""
    h = np.asarray(h8, np.float64) * expand(np.asarray(h_scale, np.float64), 1, h8.shape)
    w = np.asarray(w8, np.float64) * expand(np.asarray(w_scale, np.float64), BLOCK, w8.shape)
    return h @ w.T


def kept(z, tau=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """Ids that may be drawn from one row, ascending: temperature, then top-k, then top-p of what
    top-k kept, then min-p. Equal logits are ordered by id, the lowest first."""
    z = np.asarray(z, np.float64)
    order = np.lexsort((np.arange(z.size), -z))
    e = np.exp((z[order] - z[order[0]]) / tau)
    n = z.size
    if 0 < top_k < n:
        n = top_k
    if top_p < 1.0:
        c = np.cumsum(e[:n].astype(np.longdouble))
        n = min(n, int(np.searchsorted(c, np.longdouble(top_p) * c[-1])) + 1)
    if min_p > 0.0:
        low = math.log(min(min_p, 1.0))
        n = int(np.sum((z[order[:n]] - z[order[0]]) / tau >= low))
    return np.sort(order[:n])


def sample(z, u, tau=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """-> (token, logprob under the tempered softmax over the whole row); (-1, 0) for a row whose
    log-sum-exp is not finite."""
    z = np.asarray(z, np.float64)
    if np.isnan(z).any() or not np.isfinite(z.max()):
        return -1, 0.0
    ids = kept(z, tau, top_k, top_p, min_p)
    e = np.exp((z[ids] - z.max()) / tau)
    c = np.cumsum(e)
    j = min(int(np.sum(c <= u * c[-1])), ids.size - 1)
    t = int(ids[j])
    t0 = (z - z.max()) / tau
    return t, float(t0[t] - math.log(math.fsum(np.exp(t0))))
