"""Places of the residual stream's norm that its own tests do not reach.

Tolerances are those of test_gpu_rmsnorm.py.
"""
import numpy as np
import pytest
import torch

import test_gpu_rmsnorm as tn
from gated_delta_rule_96_amd import kda
from kda_testutil import say
from oracle import block

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF = torch.bfloat16


@pytest.mark.parametrize("rows,D,lone", [(2 * 2048 + 37, 8200, 2048), (3 * 2048 + 1, 16384, 2048), (32 * (1 << 20) + 77, 8, 900)])
def test_norm_rows_that_a_work_group_walks_on_to(rows, D, lone):
    # more rows than the forward's work-groups hold at once: 2048 rows of more than
    # 8192 channels, 32 x 2^20 of up to 64.  The same rows in a call of their own have
    # the same bits.
    say(f"norm {rows} x {D}")
    gen = torch.Generator(device="cuda").manual_seed(231)
    x = torch.randn((rows, D), dtype=BF, device="cuda", generator=gen)
    w = torch.rand(D, device="cuda", generator=gen) + 0.5
    (y8, sc), h = kda.add_rms_norm(x, x, w, fp8=True)
    y, _ = kda.add_rms_norm(x, None, w)
    for lo in ([0, rows - lone] if D == 8 else range(0, rows, lone)):
        part = x[lo:lo + lone].clone()
        (p8, psc), ph = kda.add_rms_norm(part, part, w, fp8=True)
        py, _ = kda.add_rms_norm(part, None, w)
        at = slice(lo, lo + len(part))
        assert torch.equal(y8[at].view(torch.uint8), p8.view(torch.uint8)) and torch.equal(sc[at], psc) and torch.equal(h[at], ph) and torch.equal(y[at], py)
    for m in (0, lone, rows - 1):
        n = block.rms_norm(tn.f64(x[m:m + 1]), tn.f64(w), 1e-6)
        tn.check("y", y[m:m + 1], n, 36 * U * np.abs(n), BF)
        tn.check8(y8[m:m + 1], sc[m:m + 1], block.rms_norm(tn.f64(h[m:m + 1]), tn.f64(w), 1e-6))


@pytest.mark.parametrize("rows,D", [(3, 64), (40, 520)])
def test_gradients_of_the_norm_along_themselves(rows, D):
    # x and w each along its own gradient G, d = G / max |G|: the slope sum G^2 / max
    # |G| against the oracle's central difference in 64 bits (its step of 2^-14 is off by
    # less than the differences at 2^-14 and 2^-13 are apart), within the gradients' own
    # tolerances
    r = np.random.default_rng(291)
    x, w, dy = (r.standard_normal(s).astype(np.float32).astype(np.float64) for s in ((rows, D), (D,), (rows, D)))
    got = kda.add_rms_norm_bwd(tn.dev(x), tn.dev(w), tn.dev(dy), eps=1e-6)
    dx, dw = block.rms_norm_bwd(x, w, dy, None, 1e-6)
    rn, gw = 1 / np.sqrt((x * x).mean(1, keepdims=True) + 1e-6), np.abs(dy * w)
    tx = 40 * U * rn * gw + 140 * U * np.abs(x) * rn ** 3 * (gw * np.abs(x)).mean(1, keepdims=True) + 2 * U * np.abs(dx)
    tw = (40 + rows / tn.HOLDERS + 1) * U * np.abs(dy * x * rn).sum(0)
    for n, G, tol, f in (("dx", dx, tx, lambda v: block.rms_norm(x + v, w, 1e-6)), ("dw", dw, tw, lambda v: block.rms_norm(x, w + v, 1e-6))):
        d = G / np.abs(G).max()
        slope = lambda e: float(((f(e * d) - f(-e * d)) * dy).sum() / (2 * e))
        s = slope(2.0 ** -14)
        lim = abs(s - slope(2.0 ** -13)) + float(((tol + U * np.abs(G)) * np.abs(d)).sum())
        assert lim <= 1e-3 * s and abs(float((tn.f64(got[n]) * d).sum()) - s) <= lim, n
