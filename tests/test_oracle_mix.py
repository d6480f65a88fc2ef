"""Pins of oracle/mix.py: token-by-token sums, carry across a cut, finite
differences, complex products."""
import numpy as np
import pytest

from oracle import mix


def rnd(*s, seed=0):
    return np.random.default_rng(seed).standard_normal(s)


@pytest.mark.parametrize("W", [2, 3, 4])
def test_conv_is_the_sum_over_taps(W):
    x, w, b, s0 = rnd(7, 3), rnd(3, W, seed=1), rnd(3, seed=2), rnd(W - 1, 3, seed=3)
    y, st, _, _ = mix.conv_fwd(x, w, b, s0, False)
    row = lambda t: x[t] if t >= 0 else s0[W - 1 + t]
    for t in range(7):
        assert np.allclose(y[t], b + sum(w[:, j] * row(t - (W - 1 - j)) for j in range(W)))
    assert np.array_equal(st, np.concatenate([s0, x])[-(W - 1):])


def test_conv_carry_across_a_cut():
    x, w, s0 = rnd(9, 4), rnd(4, 4, seed=1), rnd(3, 4, seed=2)
    y, st, _, _ = mix.conv_fwd(x, w, None, s0, True)
    for cut in (0, 1, 2, 5, 9):
        y1, s1, _, _ = mix.conv_fwd(x[:cut], w, None, s0, True)
        y2, s2, _, _ = mix.conv_fwd(x[cut:], w, None, s1, True)
        assert np.allclose(np.concatenate([y1, y2]), y) and np.array_equal(s2, st)


def _diff(f, v, i, h=1e-6):
    a, b = v.copy(), v.copy()
    a.flat[i] += h
    b.flat[i] -= h
    return (f(a) - f(b)) / (2 * h)


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("T", [1, 2, 6])
def test_conv_gradients_by_differences(silu, T):
    x, w, b, s0, dy, dst = rnd(T, 2), rnd(2, 4, seed=1), rnd(2, seed=2), rnd(3, 2, seed=3), rnd(T, 2, seed=4), rnd(3, 2, seed=5)
    dx, dw, db, ds0, _ = mix.conv_bwd(x, w, b, s0, dy, dst, silu)

    def loss(x=x, w=w, b=b, s0=s0):
        y, st, _, _ = mix.conv_fwd(x, w, b, s0, silu)
        return (y * dy).sum() + (st * dst).sum()
    for name, v, g in (("x", x, dx), ("w", w, dw), ("b", b, db), ("s0", s0, ds0)):
        for i in range(v.size):
            assert np.isclose(_diff(lambda u: loss(**{name: u}), v, i), g.flat[i], atol=1e-7), (name, i)


@pytest.mark.parametrize("inter", [False, True])
def test_turn_is_a_complex_product(inter):
    x, ang = rnd(5, 3, 16), rnd(5, 4, seed=1)
    y = mix.turn(x, np.cos(ang)[:, None], np.sin(ang)[:, None], inter)
    a, b = mix._halves(x, 8, inter)
    z = (a + 1j * b) * np.exp(1j * ang)[:, None]
    ya, yb = mix._halves(y, 8, inter)
    assert np.allclose(ya, z.real) and np.allclose(yb, z.imag) and np.array_equal(y[..., 8:], x[..., 8:])
    assert np.allclose((y * y).sum(-1), (x * x).sum(-1))
    assert np.allclose(mix.turn(y, np.cos(ang)[:, None], -np.sin(ang)[:, None], inter), x)


@pytest.mark.parametrize("rms", [False, True])
def test_norm_lengths(rms):
    x = rnd(4, 2, 8)
    n = mix.qk_fwd(x, None, None, None, rms, False, eps=0.0)
    assert np.allclose((n * n).sum(-1), 8 if rms else 1) and np.allclose(mix.qk_fwd(3 * x, None, None, None, rms, False, eps=0.0), n)
    assert not mix.qk_fwd(0 * x, None, None, None, rms, False).any()


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("inter", [False, True])
def test_norm_gradients_by_differences(rms, inter):
    x, w, ang, dy = rnd(2, 2, 8), rnd(8, seed=1), rnd(2, 2, seed=2), rnd(2, 2, 8, seed=3)
    c, s = np.cos(ang), np.sin(ang)
    dx, dw = mix.qk_bwd(x, w, c, s, dy, rms, inter)
    for i in range(x.size):
        assert np.isclose(_diff(lambda u: (mix.qk_fwd(u, w, c, s, rms, inter) * dy).sum(), x, i), dx.flat[i], atol=1e-6)
    for i in range(w.size):
        assert np.isclose(_diff(lambda u: (mix.qk_fwd(x, u, c, s, rms, inter) * dy).sum(), w, i), dw.flat[i], atol=1e-6)


def _scan_case(T, H, G, dk, dv, seed=3):
    r = np.random.default_rng(seed)
    return dict(x=r.standard_normal((T, H, dv)), raw=r.standard_normal((T, H)), A=-r.uniform(0.5, 4, H), Bm=r.standard_normal((T, G, dk)),
                Cm=r.standard_normal((T, G, dk)), h0=r.standard_normal((H, dk, dv)), D=r.standard_normal(H), bias=r.standard_normal(H))


def test_scan_is_the_lower_triangular_product():
    c = _scan_case(9, 4, 2, 3, 5)
    y, ht, size, _ = mix.ssm_seq(**c, soft=True)
    dt = np.log1p(np.exp(c["raw"] + c["bias"]))
    for h in range(4):
        cum = np.cumsum(dt[:, h] * c["A"][h])
        M = np.tril((c["Cm"][:, h // 2] @ c["Bm"][:, h // 2].T) * np.exp(np.minimum(cum[:, None] - cum[None], 0))) * dt[:, h]
        want = M @ c["x"][:, h] + np.exp(cum)[:, None] * (c["Cm"][:, h // 2] @ c["h0"][h]) + c["D"][h] * c["x"][:, h]
        assert np.allclose(y[:, h], want)
    assert (size >= np.abs(y) - 1e-12).all()


def test_scan_carry_and_identity():
    c = _scan_case(8, 2, 1, 4, 4)
    y, ht, _, _ = mix.ssm_seq(**c)
    cut = lambda lo, hi, h0: mix.ssm_seq(**{**c, "x": c["x"][lo:hi], "raw": c["raw"][lo:hi], "Bm": c["Bm"][lo:hi], "Cm": c["Cm"][lo:hi], "h0": h0})
    y1, h1, _, _ = cut(0, 3, c["h0"])
    y2, h2, _, _ = cut(3, 8, h1)
    assert np.allclose(np.concatenate([y1, y2]), y) and np.allclose(h2, ht)
    z = dict(c, raw=np.zeros((8, 2)), bias=None)
    assert np.allclose(mix.ssm_seq(**z)[1], c["h0"])   # steps of size zero leave the state


@pytest.mark.parametrize("soft", [False, True])
def test_scan_gradients_by_differences(soft):
    c = _scan_case(5, 4, 2, 2, 3)
    if not soft:
        c["raw"], c["bias"] = np.abs(c["raw"]), None
    dy, dht = rnd(5, 4, 3, seed=8), rnd(4, 2, 3, seed=9)
    g = mix.ssm_seq_bwd(**{k: v for k, v in c.items()}, dy=dy, dht=dht, soft=soft)

    def loss(**kw):
        y, ht, _, _ = mix.ssm_seq(**{**c, **kw}, soft=soft)
        return (y * dy).sum() + (ht * dht).sum()
    for n, gn in (("x", "dx"), ("raw", "ddt"), ("A", "dA"), ("Bm", "dB"), ("Cm", "dC"), ("D", "dD"), ("bias", "ddt_bias"), ("h0", "dh0")):
        if c[n] is None:
            continue
        for i in range(c[n].size):
            assert np.isclose(_diff(lambda u: loss(**{n: u}), c[n], i), g[gn].flat[i], rtol=1e-5, atol=1e-6), (n, i)
        assert (g[gn + "|"] >= np.abs(g[gn]) - 1e-9).all()
