"""GPU parity of the residual stream's norm (kda_add_rms_norm and its
gradients) against the fp64 oracle (oracle/block.py).

Tolerances, per element, u = 2^-24.  A mean of squares: two roundings a term,
at most 32 additions in a lane, 6 lane steps, 16 waves: 56 u, half of it in the
root; with the root, the reciprocal, eps and the products n is off by 36 u |n|,
and by the output's rounding h (finfo.eps / 2).  h itself is one rounded sum:
equal.  8 bits: scales off by 38 u; a value by half a step of its own (2^-4
relative, 2^-10 of the scale below the type's normal range) and 45 u |n|.
Backward: mean(w dy h) is off by 66 u m1, m1 = mean |w dy h|; dx = r (w dy - h r^2
mean) then by r 40 u |w dy| + 140 u |h| r^3 m1, and u for the sum with dh.  dw
sums k rows of a holder in fp32 and the holders in 64 bits: (40 + k) u sum |dy u|.
"""
import numpy as np
import pytest
import torch

from gated_delta_rule_96_amd import kda
from kda_testutil import cast, say
from oracle import block

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-6
BF, F32 = torch.bfloat16, torch.float32
HOLDERS = 512   # work-groups of the backward at most: rows a holder sums


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def dev(a, dtype=F32):
    return cast(a, dtype).cuda()


def check(name, got, want, tol, dtype):
    h = torch.finfo(dtype).eps / 2
    lim = tol * (1 + h) + h * np.abs(want)
    bad = ~(np.abs(f64(got) - want) <= lim)
    assert not bad.any(), (name, int(bad.sum()), float(np.max(np.abs(f64(got) - want) / (lim + 1e-300))))


def slice_of(a, dtype, pad):
    """The rows as a slice of a wider tensor."""
    wide = torch.full((a.shape[0], a.shape[1] + pad), float("nan"), dtype=dtype, device="cuda")
    wide[:, :a.shape[1]] = dev(a, dtype)
    return wide[:, :a.shape[1]]


def check8(y8, scale, n):
    """8-bit rows and scales against the 64-bit norm."""
    top = block.block_max(n) / block.E4M3
    top[top == 0] = 1
    assert np.all(np.abs(f64(scale) - top) <= 38 * U * top)
    s = block.spread(f64(scale), n.shape[1])
    q = f64(y8.float())
    lim = np.maximum(2.0 ** -4 * np.abs(n), 2.0 ** -10 * s) * (1 + 50 * U) + 45 * U * np.abs(n)
    assert np.all(np.abs(q * s - n) <= lim)


WIDTHS = [8, 64, 120, 512, 520, 1024, 2048, 2056, 4096, 4360, 8192, 8200, 16384]


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("dtype,res", [(BF, BF), (BF, F32), (BF, None), (F32, F32), (F32, None)])
def test_forward(dtype, res, D):
    say(f"norm {dtype} res {res} D={D}")
    r = np.random.default_rng(D)
    for rows, pad in ((1, 0), (5, 8), (67, 0)):
        x = slice_of(r.standard_normal((rows, D)) * np.exp(r.standard_normal(D)), dtype, pad)
        s = slice_of(3 * r.standard_normal((rows, D)), res, 2 * pad) if res else None
        w = dev(1 + 0.2 * r.standard_normal(D)) if rows != 5 else None
        y, h = kda.add_rms_norm(x, s, w, eps=EPS)
        (y8, scale), h8 = kda.add_rms_norm(x, s, w, eps=EPS, fp8=True)
        torch.cuda.synchronize()
        if res:
            want = (x.float() + s.float()).to(res)
            assert torch.equal(h, want) and torch.equal(h8, want)
        else:
            want = x
            assert h is None and h8 is None
        n = block.rms_norm(f64(want), f64(w), EPS)
        check("y", y, n, 36 * U * np.abs(n), dtype)
        assert y8.dtype == torch.float8_e4m3fn and scale.shape == (rows, (D + 127) // 128)
        check8(y8, scale, n)


@pytest.mark.parametrize("D", [8, 200, 1024, 2048, 4096, 6400, 8200, 16384])
@pytest.mark.parametrize("dtype,gtype", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
def test_gradients(dtype, gtype, D):
    say(f"norm gradients {dtype} {gtype} D={D}")
    r = np.random.default_rng(D + 1)
    for rows, weight, skip in ((1, True, True), (9, False, True), (1500 if D < 4096 else 700, True, False)):
        h = slice_of(2 * r.standard_normal((rows, D)), dtype, 8 if rows == 9 else 0)
        dy, dh = dev(r.standard_normal((rows, D)), gtype), dev(r.standard_normal((rows, D)), dtype) if skip else None
        w = dev(1 + 0.2 * r.standard_normal(D)) if weight else None
        got = kda.add_rms_norm_bwd(h, w, dy, dh, eps=EPS, want_dw=True)
        again = kda.add_rms_norm_bwd(h, w, dy, dh, eps=EPS)
        torch.cuda.synchronize()
        x, g = f64(h), f64(dy)
        dx, dw = block.rms_norm_bwd(x, f64(w), g, f64(dh), EPS)
        rr = 1 / np.sqrt((x * x).mean(1, keepdims=True) + EPS)
        gw = np.abs(g * (1.0 if w is None else f64(w)))
        m1 = (gw * np.abs(x)).mean(1, keepdims=True)
        tol = 40 * U * rr * gw + 140 * U * np.abs(x) * rr ** 3 * m1 + 2 * U * (np.abs(dx) + (0 if dh is None else np.abs(f64(dh))))
        check("dx", got["dx"], dx, tol, dtype)
        check("dw", got["dw"], dw, (40 + rows / HOLDERS + 1) * U * np.abs(g * x * rr).sum(0), F32)
        assert torch.equal(got["dx"], again["dx"])
        assert again["dw"] is None if w is None else torch.equal(got["dw"], again["dw"])


def test_gradient_of_the_forward_against_differences():
    # the forward's own slope in fp32: a central difference with step e is off by
    # e^2 f''' / 6 and by its values' rounding, 36 u sum |n dy| / e each
    r = np.random.default_rng(5)
    x, w, dy, d = (dev(r.standard_normal(s)) for s in ((3, 64), (64,), (3, 64), (3, 64)))
    e = 2.0 ** -7
    f = lambda t: float((kda.add_rms_norm(t, None, w)[0].double() * dy.double()).sum())
    slope = (f(x + e * d) - f(x - e * d)) / (2 * e)
    got = float((kda.add_rms_norm_bwd(x, w, dy)["dx"].double() * d.double()).sum())
    size = float((dy.abs() * w.abs()).double().sum() * 4)
    assert abs(slope - got) <= 40 * e * e * size + 2 * 36 * U * size / e


def test_in_place_and_leading_sizes():
    r = np.random.default_rng(6)
    x, s = dev(r.standard_normal((2, 7, 256)), BF), dev(r.standard_normal((2, 7, 256)))
    y, h = kda.add_rms_norm(x, s)
    s2 = s.clone()
    y2, h2 = kda.add_rms_norm(x, s2, sum_out=s2)
    assert h2 is s2 and torch.equal(h, s2) and torch.equal(y, y2) and y.shape == x.shape
    (y8, sc), _ = kda.add_rms_norm(x, s, fp8=True)
    assert y8.shape == x.shape and sc.shape == (2, 7, 2)
    dh = dev(r.standard_normal((2, 7, 256)))
    want = kda.add_rms_norm_bwd(h, None, y, dh)["dx"]
    got = kda.add_rms_norm_bwd(h, None, y, dh, out={"dx": dh, "dw": None})["dx"]
    assert got is dh and torch.equal(want, dh)


def test_zero_rows_blocks_and_values_that_are_not_finite():
    x = torch.zeros(4, 512, device="cuda")
    x[1, 3] = 2.0                     # three blocks of zeros
    x[2] = 1.0
    x[2, 200] = float("nan")
    x[3] = float("inf")
    y, _ = kda.add_rms_norm(x)
    (y8, s), _ = kda.add_rms_norm(x, fp8=True)
    assert not y[0].any() and not y8[0].float().any() and torch.equal(s[0], torch.ones(4, device="cuda"))
    assert torch.equal(s[1, 1:], torch.ones(3, device="cuda")) and float(y8[1, 3].float()) == 448.0
    assert torch.isnan(y[2]).all() and torch.isnan(y8[2].float()).all() and torch.isnan(y[3]).all() and torch.isnan(y8[3].float()).all()
    big = torch.full((1, 512), 1e18, device="cuda")     # squares sum to 5e38: past fp32, their mean is not
    assert torch.allclose(kda.add_rms_norm(big)[0], torch.ones_like(big))
    z = kda.add_rms_norm(x[:1], eps=0.0)[0]
    assert torch.isnan(z).all()


def test_many_rows_and_far_ones():
    # rows past the work-groups of one launch, and rows 2^24 elements apart
    r = np.random.default_rng(7)
    x = dev(r.standard_normal((9000, 64)), BF)
    y, _ = kda.add_rms_norm(x)
    assert torch.equal(y[8191:], kda.add_rms_norm(x[8191:].contiguous())[0])
    wide = torch.empty((150, 1 << 24), dtype=BF, device="cuda")
    wide[:, -72:-8] = x[:150]
    assert torch.equal(kda.add_rms_norm(wide[:, -72:-8])[0], y[:150])


def test_refusals():
    x = torch.zeros(4, 64, dtype=BF, device="cuda")
    with pytest.raises(ValueError, match="res must be"):
        kda.add_rms_norm(x, x[:2])
    with pytest.raises(kda.KDAError):
        kda.add_rms_norm(x.float(), x)           # a bf16 stream under fp32 rows
    with pytest.raises(kda.KDAError):
        kda.add_rms_norm(torch.zeros(2, 12, device="cuda"))
    with pytest.raises(kda.KDAError) as e:
        kda.add_rms_norm(x, x, out=x)
    assert e.value.status == kda.KDA_ERR_OVERLAP
    with pytest.raises(ValueError, match="sum_out"):
        kda.add_rms_norm(x, sum_out=x)
    with pytest.raises(TypeError, match="dh"):
        kda.add_rms_norm_bwd(x, None, x.clone(), x.float())


@pytest.mark.parametrize("D", [8, 24, 56, 64, 72, 128, 136, 248, 256, 264])
def test_rows_that_share_a_wave(D):
    # more and fewer rows than a work-group holds; a row that is not finite leaves
    # its neighbours alone; the gradients of rows that meet in one partial sum
    say(f"short rows D={D}")
    r = np.random.default_rng(D + 2)
    for rows in (3, 37, 2500):
        x, s, g = (dev(r.standard_normal((rows, D)), BF) for _ in range(3))
        w = dev(1 + 0.2 * r.standard_normal(D))
        (y8, sc), h = kda.add_rms_norm(x, s, w, eps=EPS, fp8=True)
        y, _ = kda.add_rms_norm(x, s, w, eps=EPS)
        n = block.rms_norm(f64(h), f64(w), EPS)
        check("y", y, n, 36 * U * np.abs(n), BF)
        check8(y8, sc, n)
        for a in (0, rows - 1):   # a row alone has the same bits
            (one8, onesc), _ = kda.add_rms_norm(x[a:a + 1], s[a:a + 1], w, eps=EPS, fp8=True)
            assert torch.equal(one8.view(torch.uint8), y8[a:a + 1].view(torch.uint8)) and torch.equal(onesc, sc[a:a + 1])
        bad = x.clone()
        bad[1, D - 1] = float("nan")
        (b8, bsc), _ = kda.add_rms_norm(bad, s, w, eps=EPS, fp8=True)
        keep = [m for m in range(rows) if m != 1]
        assert torch.isnan(b8[1].float()).all()
        assert torch.equal(b8[keep].view(torch.uint8), y8[keep].view(torch.uint8)) and torch.equal(bsc[keep], sc[keep])
        got = kda.add_rms_norm_bwd(h, w, g, None, eps=EPS)
        again = kda.add_rms_norm_bwd(h, w, g, None, eps=EPS)
        x64, g64 = f64(h), f64(g)
        dx, dw = block.rms_norm_bwd(x64, f64(w), g64, None, EPS)
        rr = 1 / np.sqrt((x64 * x64).mean(1, keepdims=True) + EPS)
        gw = np.abs(g64 * f64(w))
        m1 = (gw * np.abs(x64)).mean(1, keepdims=True)
        check("dx", got["dx"], dx, 40 * U * rr * gw + 140 * U * np.abs(x64) * rr ** 3 * m1 + 2 * U * np.abs(dx), BF)
        check("dw", got["dw"], dw, (40 + rows / HOLDERS + 1) * U * np.abs(g64 * x64 * rr).sum(0), F32)
        assert torch.equal(got["dx"], again["dx"]) and torch.equal(got["dw"], again["dw"])
