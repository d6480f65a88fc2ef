"""fp64 operators of a recurrent block -- TEST INFRASTRUCTURE ONLY.

Definitions (the standard forms; the pages define none of them):
  * norm of the residual stream: h = x + res (rounded by the caller), n = w h /
    sqrt(mean h^2 + eps);
  * scales by blocks of 128: s = max |n| / 448, 1 for a block of zeros;
  * product of rows and weights held as values with such scales;
  * gated linear recurrence: g = -c Sigmoid(r) (or r), a = exp(g), m =
    sqrt(1 - a^2) (or 1), h_t = a h_{t-1} + m Sigmoid(i) x.

Pinned by tests/test_oracle_block.py: finite differences of the gradients,
carry across a cut, closed forms, products by blocks.
"""
from __future__ import annotations

import numpy as np

BLOCK, E4M3 = 128, 448.0


def sigmoid(z):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-z))


def rms_norm(h, w, eps):
    return h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * (1.0 if w is None else w)


def rms_norm_bwd(h, w, dy, dh, eps):
    """(dx, dw); dw of a weight of ones where w is None."""
    r = 1.0 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    g = dy * (1.0 if w is None else w)
    dx = r * g - h * r ** 3 * (g * h).mean(-1, keepdims=True)
    return dx + (0.0 if dh is None else dh), (dy * h * r).sum(0)


def block_max(n):
    """Largest |n| of every 128 channels: [rows, blocks]."""
    return np.stack([np.abs(n[:, k:k + BLOCK]).max(1) for k in range(0, n.shape[1], BLOCK)], 1)


def spread(s, n, axis=-1):
    """A scale for every index from one for every block."""
    return np.take(s, np.arange(n) // BLOCK, axis=axis)


def product(a, sa, w, sw):
    """a [M,K], sa [M,KB], w [N,K], sw [NB,KB]."""
    return (a * spread(sa, a.shape[1])) @ (w * spread(spread(sw, a.shape[1]), w.shape[0], 0)).T


def lru_gates(x, r, i, c, unit):
    """g, a, m and Sigmoid(i) of every token."""
    g = r if c is None else -c * sigmoid(r)
    return g, np.exp(g), np.sqrt(-np.expm1(2 * g)) if unit else np.ones_like(g), np.ones_like(x) if i is None else sigmoid(i)


def lru_fwd(x, r, i, c, h0, unit):
    """One sequence, x [T,D] -> (y, ht)."""
    _, a, m, s = lru_gates(x, r, i, c, unit)
    u, h, y = m * s * x, np.zeros(x.shape[1]) if h0 is None else h0.copy(), np.empty_like(x)
    for t in range(x.shape[0]):
        h = a[t] * h + u[t]
        y[t] = h
    return y, h


def lru_bwd(x, r, i, c, h0, dy, dht, unit):
    """Gradients (dx, dr, di, dc, dh0) of one sequence, and dL/dh_t."""
    g, a, m, s = lru_gates(x, r, i, c, unit)
    y, _ = lru_fwd(x, r, i, c, h0, unit)
    before = np.concatenate([np.zeros((1, x.shape[1])) if h0 is None else h0[None], y])[:-1]
    lam, e = np.empty_like(x), np.zeros(x.shape[1]) if dht is None else dht.copy()
    for t in range(x.shape[0] - 1, -1, -1):
        lam[t] = dy[t] + e
        e = a[t] * lam[t]
    dg = lam * before * a
    if unit:
        with np.errstate(divide="ignore", invalid="ignore"):
            dg = dg - np.where(m > 0, lam * s * x * a * a / m, 0.0)
    sr = sigmoid(r)
    dr = dg if c is None else dg * g * sigmoid(-r)
    di = None if i is None else lam * m * x * s * sigmoid(-i)
    return lam * m * s, dr, di, None if c is None else -(dg * sr).sum(0), e, lam
