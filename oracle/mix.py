"""fp64 short convolution and head norms with rotation -- TEST INFRASTRUCTURE ONLY.

Definitions (the standard forms; the pages only say that KDA's queries and
keys are normalised, "Key claims", section 2.1):
  * convolution: z[t] = bias + sum_j w[:, j] x[t-(W-1-j)], rows before the
    first token from the state; y = z or z Sigmoid(z); the state behind the
    last token is the last W-1 rows;
  * head norm and rotation: n = w x / sqrt(sum x^2 (/ d) + eps), then channel
    pairs of the first rot channels turn by the token's angle.

Each function takes one sequence.  Pinned by tests/test_oracle_mix.py: token
by token sums, carry across a cut, finite differences of the gradients,
angles as complex products, lengths kept by a rotation.
"""
from __future__ import annotations

import numpy as np


def sigmoid(z):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-z))


def conv_fwd(x, w, bias, s0, silu):
    """x [T,D], w [D,W], bias [D] or None, s0 [W-1,D] or None -> (y, st, z, rows)
    with rows = [state, tokens]."""
    T, D = x.shape
    W = w.shape[1]
    rows = np.concatenate([np.zeros((W - 1, D)) if s0 is None else s0, x])
    z = sum(rows[j:j + T] * w[:, j] for j in range(W)) + (0.0 if bias is None else bias)
    return (z * sigmoid(z) if silu else z), rows[T:], z, rows


def conv_bwd(x, w, bias, s0, dy, dst, silu):
    """Gradients (dx, dw, dbias, ds0) and dz of conv_fwd."""
    T, _ = x.shape
    W = w.shape[1]
    _, _, z, rows = conv_fwd(x, w, bias, s0, silu)
    sg = sigmoid(z)
    dz = dy * sg * (1 + z * (1 - sg)) if silu else dy
    drows = np.zeros_like(rows)
    for j in range(W):
        drows[j:j + T] += dz * w[:, j]
    if dst is not None:
        drows[T:] += dst
    dw = np.stack([(dz * rows[j:j + T]).sum(0) for j in range(W)], 1)
    return drows[W - 1:], dw, dz.sum(0), drows[:W - 1], dz


def _halves(x, rot, inter):
    return (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])


def turn(x, cos, sin, inter):
    """x [...,d] turned by the angles cos, sin [...,rot/2]."""
    rot = 2 * cos.shape[-1]
    a, b = _halves(x, rot, inter)
    y = np.array(x, dtype=np.float64)
    ya, yb = _halves(y, rot, inter)
    ya[...], yb[...] = a * cos - b * sin, b * cos + a * sin
    return y


def _rinv(x, rms, eps):
    s = (x * x).sum(-1, keepdims=True)
    return 1.0 / np.sqrt((s / x.shape[-1] if rms else s) + eps)


def qk_fwd(x, w, cos, sin, rms, inter, eps=1e-6):
    """x [T,H,d]; cos, sin [T,rot/2] of the tokens or None."""
    n = x * _rinv(x, rms, eps) * (1.0 if w is None else w)
    return n if cos is None else turn(n, cos[:, None], sin[:, None], inter)


def qk_bwd(x, w, cos, sin, dy, rms, inter, eps=1e-6):
    """(dx, dw) of qk_fwd; dw of a weight of ones where w is None."""
    dn = dy if cos is None else turn(dy, cos[:, None], -sin[:, None], inter)
    r = _rinv(x, rms, eps)
    dw = (dn * x * r).sum((0, 1))
    g = dn * (1.0 if w is None else w)
    dot = (g * x).sum(-1, keepdims=True) / (x.shape[-1] if rms else 1)
    return g * r - x * dot * r ** 3, dw


def softplus(x):
    return np.logaddexp(x, 0.0)


def ssm_seq(x, raw, A, Bm, Cm, h0=None, D=None, bias=None, soft=False):
    """One sequence of the scan token by token: x [T,H,dv], raw [T,H], Bm, Cm
    [T,G,dk], h0 [H,dk,dv] -> (y, ht, size) with size the same recurrence on
    absolute values (what the outputs' roundings are relative to)."""
    T, H, dv = x.shape
    G, dk = Bm.shape[1:]
    dt = raw + (0.0 if bias is None else bias)
    dt = softplus(dt) if soft else dt
    b, c = np.repeat(Bm, H // G, 1), np.repeat(Cm, H // G, 1)
    S = np.zeros((H, dk, dv)) if h0 is None else np.array(h0, dtype=np.float64)
    Z = np.abs(S)
    y, size = np.zeros((T, H, dv)), np.zeros((T, H, dv))
    for t in range(T):
        e = np.exp(dt[t] * A)[:, None, None]
        S = S * e + (dt[t][:, None] * b[t])[:, :, None] * x[t][:, None]
        Z = Z * e + (np.abs(dt[t])[:, None] * np.abs(b[t]))[:, :, None] * np.abs(x[t])[:, None]
        y[t] = (S * c[t][:, :, None]).sum(1)
        size[t] = (Z * np.abs(c[t])[:, :, None]).sum(1)
        if D is not None:
            y[t] += D[:, None] * x[t]
            size[t] += np.abs(D[:, None] * x[t])
    return y, S, size, Z


def ssm_seq_bwd(x, raw, A, Bm, Cm, dy, h0=None, dht=None, D=None, bias=None, soft=False):
    """Gradients of ssm_seq, token by token against the sequence: a dict of dx,
    ddt, dA, dB, dC, dD, ddt_bias, dh0, and under the same names with a "|"
    the same sums over absolute values (what roundings are relative to)."""
    T, H, dv = x.shape
    G, dk = Bm.shape[1:]
    v = raw + (0.0 if bias is None else bias)
    dt = softplus(v) if soft else v
    sg = sigmoid(v) if soft else np.ones_like(v)
    b, c = np.repeat(Bm, H // G, 1), np.repeat(Cm, H // G, 1)
    S = np.zeros((T + 1, H, dk, dv))
    Z = np.zeros_like(S)
    if h0 is not None:
        S[0], Z[0] = h0, np.abs(h0)
    e = np.exp(dt * A)[..., None, None]
    for t in range(T):
        S[t + 1] = S[t] * e[t] + (dt[t][:, None] * b[t])[:, :, None] * x[t][:, None]
        Z[t + 1] = Z[t] * e[t] + (np.abs(dt[t])[:, None] * np.abs(b[t]))[:, :, None] * np.abs(x[t])[:, None]
    dS = np.zeros((H, dk, dv)) if dht is None else np.array(dht, dtype=np.float64)
    dZ = np.abs(dS)
    o = {n: np.zeros(s) for n, s in (("dx", x.shape), ("ddt", raw.shape), ("dA", (H,)), ("dB", b.shape), ("dC", c.shape), ("dD", (H,)),
                                     ("ddt_bias", (H,)))}
    o.update({n + "|": np.zeros_like(a) for n, a in list(o.items())})
    for sgn, SS, dd, f in (("", S, dS, lambda a: a), ("|", Z, dZ, np.abs)):
        for t in range(T - 1, -1, -1):
            bb, cc, xx, yy, tt = f(b[t]), f(c[t]), f(x[t]), f(dy[t]), f(dt[t])
            o["dC" + sgn][t] = (SS[t + 1] * yy[:, None]).sum(2)
            dd = dd + cc[:, :, None] * yy[:, None]
            o["dx" + sgn][t] = tt[:, None] * (dd * bb[:, :, None]).sum(1) + (0 if D is None else f(D)[:, None] * yy)
            o["dB" + sgn][t] = tt[:, None] * (dd * xx[:, None]).sum(2)
            da = (dd * SS[t] * e[t]).sum((1, 2))
            d = f(A) * da + (dd * bb[:, :, None] * xx[:, None]).sum((1, 2))
            o["dA" + sgn] += tt * da
            o["ddt" + sgn][t] = d * sg[t]
            o["ddt_bias" + sgn] += d * sg[t]
            o["dD" + sgn] += (xx * yy).sum(1)
            dd = dd * e[t]
        o["dh0" + sgn] = dd
    for n in ("dB", "dC", "dB|", "dC|"):
        o[n] = o[n].reshape(T, G, H // G, dk).sum(2)
    return o
