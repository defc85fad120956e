"""Training oracle: layer norm, the global gradient norm with the clip, and
PatchGroupNorm's backward pass, in float64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

Plain definitions, written from the formulas; the
caller rounds results once into the storage type.  Where a call takes a
statistic as an input (mean, rstd of the layer norm's backward pass), so do
these functions.
"""
from typing import List, Optional, Sequence, Tuple

import numpy as np


def layer_norm(h: np.ndarray, gamma, beta, eps: float) -> Tuple[np.ndarray, np.ndarray, np.ndarray]:
    """(y, mean, rstd) of the rows of ``h`` [rows, cols]."""
    h = np.asarray(h, dtype=np.float64)
    n = h.shape[1]
    mean = h.sum(axis=1) / n
    var = ((h - mean[:, None]) ** 2).sum(axis=1) / n
    rstd = 1.0 / np.sqrt(var + eps)
    y = (h - mean[:, None]) * rstd[:, None]
    if gamma is not None:
        y = y * np.asarray(gamma, dtype=np.float64)
    if beta is not None:
        y = y + np.asarray(beta, dtype=np.float64)
    return y, mean, rstd


def layer_norm_backward(dy, x, mean, rstd, gamma, dtotal=None) -> Tuple[np.ndarray, np.ndarray, np.ndarray]:
    """(dx, dgamma, dbeta) with the given row statistics."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    mean, rstd = np.asarray(mean, np.float64)[:, None], np.asarray(rstd, np.float64)[:, None]
    n = x.shape[1]
    xhat = (x - mean) * rstd
    g = dy if gamma is None else dy * np.asarray(gamma, np.float64)
    dx = rstd * (g - g.sum(1, keepdims=True) / n - xhat * ((g * xhat).sum(1, keepdims=True) / n))
    if dtotal is not None:
        dx = dx + np.asarray(dtotal, np.float64)
    return dx, (dy * xhat).sum(0), dy.sum(0)


def grad_norm(grads: Sequence[np.ndarray]) -> float:
    return float(np.sqrt(sum(float((np.asarray(g, np.float64) ** 2).sum()) for g in grads)))


def clip_factor(norm: float, max_norm: float) -> float:
    return min(1.0, max_norm / (norm + 1e-6))


def silu_grad(z: np.ndarray) -> np.ndarray:
    """Derivative of z / (1 + exp(-z))."""
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-z))
    return s * (1.0 + z * (1.0 - s))


def group_norm_backward(dys: Sequence[np.ndarray], xs: Sequence[np.ndarray], G: int, gamma, beta, eps: float,
                        silu: bool, stats: Optional[Tuple[np.ndarray, np.ndarray]] = None
                        ) -> Tuple[List[np.ndarray], np.ndarray, np.ndarray]:
    """(dx of every patch, dgamma, dbeta) of the unsharded GroupNorm (+ SiLU)
    whose input and output gradient are given patch by patch.  ``stats``: the
    pooled (mean, rstd) [N, G]; computed when None."""
    N, C = xs[0].shape[:2]
    cg = C // G
    gam = np.ones(C) if gamma is None else np.asarray(gamma, np.float64)
    bet = np.zeros(C) if beta is None else np.asarray(beta, np.float64)
    dxs = [np.empty(x.shape, np.float64) for x in xs]
    dgamma, dbeta = np.zeros(C), np.zeros(C)
    for n in range(N):
        for g in range(G):
            chans = range(g * cg, (g + 1) * cg)
            count = sum(x[n, c].size for x in xs for c in chans)
            if stats is None:
                allx = np.concatenate([np.asarray(x[n, c], np.float64).ravel() for x in xs for c in chans])
                mu = allx.sum() / count
                rstd = 1.0 / np.sqrt(((allx - mu) ** 2).sum() / count + eps)
            else:
                mu, rstd = float(stats[0][n, g]), float(stats[1][n, g])
            c1 = c2 = 0.0
            dz = {}
            for p, (x, dy) in enumerate(zip(xs, dys)):
                for c in chans:
                    xh = (np.asarray(x[n, c], np.float64) - mu) * rstd
                    d = np.asarray(dy[n, c], np.float64)
                    if silu:
                        d = d * silu_grad(xh * gam[c] + bet[c])
                    dz[p, c] = (d, xh)
                    dbeta[c] += d.sum()
                    dgamma[c] += (d * xh).sum()
                    c1 += gam[c] * d.sum()
                    c2 += gam[c] * (d * xh).sum()
            for (p, c), (d, xh) in dz.items():
                dxs[p][n, c] = rstd * (gam[c] * d - c1 / count - xh * (c2 / count))
    return dxs, dgamma, dbeta
