"""The gradient of a recurrent block (norm of the residual stream, projection,
convolution, gated linear recurrence) against differences of the whole chain."""
import numpy as np
import pytest
import torch

import test_gpu_lru as tl
from gated_delta_rule_96_amd import kda
from kda_testutil import cast
from oracle import block, mix

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
F32 = torch.float32


def test_gradient_of_a_block_along_itself():
    # Norm, projection, convolution and recurrence: the gradient of the stream
    # along itself against the oracle's central difference of the whole chain (in
    # 64 bits; its step of 2^-12 is off by less than the differences at 2^-12 and
    # 2^-11 are apart).  The GPU's gradient: a path passes at most 350 tokens of 14
    # roundings, two sums of 130 terms and some 200 more, 5400 u of the sums of
    # absolute values A of the gradient, and as much again from the forward's
    # values: 2^-10 A.
    lens, D, E, W, EPS = [90, 260], 128, 64, 4, 1e-6
    r = np.random.default_rng(221)
    f = lambda a: a.astype(np.float32).astype(np.float64)
    T, cu = sum(lens), tl.cuts(lens)
    h, w, wp = f(2 * r.standard_normal((T, D))), f(1 + 0.2 * r.standard_normal(D)), f(r.standard_normal((3 * E, D)) / np.sqrt(D))
    cw, cb, s0, c = f(r.uniform(-0.7, 0.7, (E, W))), f(r.uniform(-0.5, 0.5, E)), f(r.standard_normal((2, W - 1, E))), f(-np.log(r.uniform(0.5, 0.999, E)))
    h0, dout, dht, dh = f(r.standard_normal((2, E))), f(r.standard_normal((T, E))), f(r.standard_normal((2, E))), f(r.standard_normal((T, D)))

    def loss(h):
        p, s = block.rms_norm(h, w, EPS) @ wp.T, 0.0
        for n, (lo, hi) in enumerate(zip(cu, cu[1:])):
            xc = mix.conv_fwd(p[lo:hi, :E], cw, cb, s0[n], True)[0]
            y, ht = block.lru_fwd(xc, p[lo:hi, E:2 * E], p[lo:hi, 2 * E:], c, h0[n], True)
            s += (y * dout[lo:hi]).sum() + (ht * dht[n]).sum()
        return s
    # the gradient and its sums of absolute values
    p, dp, ap = block.rms_norm(h, w, EPS) @ wp.T, np.empty((T, 3 * E)), np.empty((T, 3 * E))
    for n, (lo, hi) in enumerate(zip(cu, cu[1:])):
        a, rr, ii = np.split(p[lo:hi], 3, 1)
        xc = mix.conv_fwd(a, cw, cb, s0[n], True)[0]
        dx, dr, di, _, _, _ = block.lru_bwd(xc, rr, ii, c, h0[n], dout[lo:hi], dht[n], True)
        dp[lo:hi] = np.concatenate([mix.conv_bwd(a, cw, cb, s0[n], dx, None, True)[0], dr, di], 1)
        g, dec, m, si = block.lru_gates(xc, rr, ii, c, True)
        u, L, H, e, s = np.abs(m * si * xc), np.empty_like(a), np.empty_like(a), np.abs(dht[n]), np.abs(h0[n])
        for t in range(hi - lo):
            H[t] = s
            s = dec[t] * s + u[t]
        for t in range(hi - lo - 1, -1, -1):
            L[t] = np.abs(dout[lo + t]) + e
            e = dec[t] * L[t]
        size = L * (dec * H + si * np.abs(xc) * dec * dec / m)
        adx = 1.1 * L * m * si   # (a convolution's SiLU has slopes of at most 1.1)
        rows = np.concatenate([adx, np.zeros((W - 1, E))])
        ap[lo:hi] = np.concatenate([sum(np.abs(cw[:, W - 1 - j]) * rows[j:j + hi - lo] for j in range(W)),
                                    size * np.abs(g) * block.sigmoid(-rr), L * m * si * np.abs(xc) * block.sigmoid(-ii)], 1)
    G = block.rms_norm_bwd(h, w, dp @ wp, None, EPS)[0]
    rn, ag = 1 / np.sqrt((h * h).mean(1, keepdims=True) + EPS), np.abs(w) * (ap @ np.abs(wp))
    A = rn * ag + np.abs(h) * rn ** 3 * (ag * np.abs(h)).mean(1, keepdims=True)
    d, step = G / np.abs(G).max(), lambda e: (loss(h + e * d) - loss(h - e * d)) / (2 * e)
    slope, exact = step(2.0 ** -12), float((G * d).sum())
    far = abs(step(2.0 ** -11) - slope)
    assert abs(slope - exact) <= far + 1e-9 * exact and far <= 1e-4 * exact
    # the same on the GPU
    v = lambda a, *s: cast(a, F32).cuda().view(*s) if s else cast(a, F32).cuda()
    y, _ = kda.add_rms_norm(v(h, 1, T, D), None, v(w), eps=EPS)
    a, rr, ii = (y @ v(wp).t()).split(E, -1)
    xc, _ = kda.conv_fwd(a, v(cw), v(cb), v(s0), cu_seqlens=cu)
    g = kda.lru_bwd(xc, rr, ii, v(c), v(dout, 1, T, E), v(h0), v(dht), cu_seqlens=cu)
    gc = kda.conv_bwd(a, v(cw), v(cb), g["dx"], v(s0), cu_seqlens=cu)
    dy = torch.cat([gc["dx"], g["dr"], g["di"]], -1) @ v(wp)
    gn = kda.add_rms_norm_bwd(v(h, 1, T, D), v(w), dy, None, eps=EPS)
    both = kda.add_rms_norm_bwd(v(h, 1, T, D), v(w), dy, v(dh, 1, T, D), eps=EPS)
    got = tl.f64(gn["dx"])[0]
    lim = 2.0 ** -10 * float((np.abs(d) * A).sum())
    assert lim <= 0.1 * exact, (lim, exact)
    assert abs(float((got * d).sum()) - slope) <= lim + far
    assert np.all(np.abs(got - G) <= 2.0 ** -10 * A)
    # the gradient that passes the norm joins with one rounding, of the sum or of both
    assert np.all(np.abs(tl.f64(both["dx"])[0] - (got + dh)) <= U * (np.abs(got) + np.abs(got + dh)) + 2.0 ** -133)
