"""GPU parity of the head norms with the position rotation (kda_qk_norm_rope
and its gradients) against the fp64 oracle (oracle/mix.py).

Tolerances, per element, u = 2^-24, rotated pairs (a, b).  The sum of squares
over d terms (8 in a lane, at most 6 lane steps) has relative error at most 14
u, its root half of that; with the reciprocal root, the weights and x: n is
off by 14 u |n|.  A rotation adds 3 roundings of |a| + |b|: |y_err| <= 18 u
(|n_a| + |n_b|), h |y| for the output's rounding (h = finfo.eps / 2).
Backward: dn is off by 3 u (|g_a| + |g_b|); the dot product over d terms by
(14 + 3 + 3) u sum |g w x|; dx = g w r - x dot r^3 (/ d): off by 30 u (|g| |w|
r + |x| r^3 sum |g w x| (/ d)) with |g| the pair's size.  dw sums R rows per
channel: the terms' 25 u, and at most 40 + R / 1024 additions.
"""
import numpy as np
import pytest
import torch

from gated_delta_rule_96_amd import kda
from kda_testutil import cast, say
from oracle import mix

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DTYPES = [torch.float32, torch.bfloat16]


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def make(B, T, Hq, Hk, d, rot, dtype, seed, weight=True, far=0, pad=0):
    r = np.random.default_rng(seed)
    wide = cast(1.5 * r.standard_normal((B, T, (Hq + Hk) * d + pad)), dtype).cuda()
    q, k = wide[..., :Hq * d].unflatten(2, (Hq, d)), wide[..., Hq * d:(Hq + Hk) * d].unflatten(2, (Hk, d))
    if not pad:
        q, k = q.contiguous(), k.contiguous()
    c = dict(q=q, k=k, wq=None, wk=None, cos=None, sin=None, pos=None)
    if weight:
        c["wq"], c["wk"] = (cast(1 + 0.2 * r.standard_normal(d), torch.float32).cuda() for _ in range(2))
    if rot:
        n = far + T + 3
        ang = np.arange(n)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
        c["cos"], c["sin"] = cast(np.cos(ang), torch.float32).cuda(), cast(np.sin(ang), torch.float32).cuda()
        c["pos"] = torch.from_numpy(r.integers(0, n, (B, T)).astype(np.int32)).cuda()
    c["dq"], c["dk"] = cast(r.standard_normal((B, T, Hq, d)), dtype).cuda(), cast(r.standard_normal((B, T, Hk, d)), dtype).cuda()
    return c


def table(c):
    if c["cos"] is None:
        return None, None
    at = c["pos"].cpu().numpy().reshape(-1)
    return f64(c["cos"])[at], f64(c["sin"])[at]


def pair_size(x, rot, inter):
    """|a| + |b| of the pair a channel is in (|x| outside the rotation)."""
    y = np.abs(x)
    if rot:
        a, b = mix._halves(y, rot, inter)
        s = a + b
        a[...] = s
        b[...] = s
    return y


def check(name, got, want, tol, dtype):
    h = torch.finfo(dtype).eps / 2
    lim = tol * (1 + h) + h * np.abs(want)
    bad = ~(np.abs(f64(got) - want) <= lim)
    assert not bad.any(), (name, int(bad.sum()), float(np.max(np.abs(f64(got) - want) / (lim + 1e-300))))


SHAPES = [(1, 1, 1, 1, 8, 0), (2, 3, 4, 2, 64, 64), (1, 17, 32, 8, 128, 64), (3, 5, 3, 1, 96, 16), (1, 9, 2, 2, 192, 96), (2, 4, 5, 5, 256, 256),
          (1, 3, 1, 1, 512, 128), (1, 300, 16, 16, 128, 128), (1, 2, 1, 3, 24, 24)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("mode", ["l2", "rms"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("B,T,Hq,Hk,d,rot", SHAPES)
def test_fwd_and_gradients(dtype, mode, inter, B, T, Hq, Hk, d, rot):
    say(f"qk {dtype} {mode} inter={inter} B={B} T={T} Hq={Hq} Hk={Hk} d={d} rot={rot}")
    rms = mode == "rms"
    c = make(B, T, Hq, Hk, d, rot, dtype, 21, weight=d != 96, pad=0 if d == 64 else 16)
    cos, sin = table(c)
    kw = dict(cos=c["cos"], sin=c["sin"], pos=c["pos"], mode=mode, interleaved=inter)
    qo, ko = kda.qk_norm_rope(c["q"], c["k"], c["wq"], c["wk"], **kw)
    torch.cuda.synchronize()
    for n, out, H in (("q", qo, Hq), ("k", ko, Hk)):
        x, w = f64(c[n]).reshape(B * T, H, d), f64(c["w" + n])
        want = mix.qk_fwd(x, w, cos, sin, rms, inter)
        size = pair_size(mix.qk_fwd(x, w, None, None, rms, inter), rot, inter)
        check(n, out.reshape(B * T, H, d), want, 18 * U * size, dtype)
    for gtype in ([dtype] if dtype == torch.float32 else [dtype, torch.float32]):
        g = kda.qk_norm_rope_bwd(c["q"], c["k"], c["dq"].to(gtype), c["dk"].to(gtype), c["wq"], c["wk"], **kw)
        again = kda.qk_norm_rope_bwd(c["q"], c["k"], c["dq"].to(gtype), c["dk"].to(gtype), c["wq"], c["wk"], **kw)
        torch.cuda.synchronize()
        for n, H in (("q", Hq), ("k", Hk)):
            x, w, dy = f64(c[n]).reshape(B * T, H, d), f64(c["w" + n]), f64(c["d" + n]).reshape(B * T, H, d)
            dx, dw = mix.qk_bwd(x, w, cos, sin, dy, rms, inter)
            r = mix._rinv(x, rms, 1e-6)
            gs, ww = pair_size(dy, rot, inter), 1.0 if w is None else np.abs(w)
            sq = (gs * ww * np.abs(x)).sum(-1, keepdims=True) / (d if rms else 1)
            check("d" + n, g["d" + n].reshape(B * T, H, d), dx, 30 * U * (gs * ww * r + np.abs(x) * r ** 3 * sq), dtype)
            if w is None:
                assert g["dw" + n] is None
            else:
                check("dw" + n, g["dw" + n], dw, (25 + 40 + B * T * H / 1024) * U * (gs * np.abs(x) * r).sum((0, 1)), torch.float32)
        for k in g:
            assert g[k] is None or torch.equal(g[k], again[k])


def test_positions_without_a_list_and_far_ones():
    c = make(2, 6, 2, 1, 64, 64, torch.bfloat16, 22, far=5000)
    want = kda.qk_norm_rope(c["q"], c["k"], cos=c["cos"], sin=c["sin"], pos=(5000 + torch.arange(6, dtype=torch.int32, device="cuda")).repeat(2, 1))
    got = kda.qk_norm_rope(c["q"], c["k"], cos=c["cos"], sin=c["sin"], pos0=5000)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    with pytest.raises(kda.KDAError):
        kda.qk_norm_rope(c["q"], c["k"], cos=c["cos"], sin=c["sin"], pos0=5004)


def test_position_outside_the_table_is_nan_and_nothing_else():
    c = make(1, 4, 2, 1, 64, 32, torch.float32, 23)
    pos = torch.tensor([[0, -1, c["cos"].shape[0], 2]], dtype=torch.int32, device="cuda")
    q, k = kda.qk_norm_rope(c["q"], c["k"], cos=c["cos"], sin=c["sin"], pos=pos)
    for t in (q, k):
        assert torch.isnan(t[0, 1:3, :, :32]).all() and torch.isfinite(t[0, 1:3, :, 32:]).all() and torch.isfinite(t[0, [0, 3]]).all()


def test_zero_rows_and_rows_of_the_largest_values():
    q = torch.zeros(1, 2, 1, 64, device="cuda")
    q[0, 1] = 3e18
    o, none = kda.qk_norm_rope(q, None, mode="rms")
    assert none is None and not o[0, 0].any() and torch.allclose(o[0, 1], torch.ones(1, 64, device="cuda"))
    g = kda.qk_norm_rope_bwd(q, None, torch.ones_like(q), None, mode="rms")
    assert torch.isfinite(g["dq"]).all() and torch.allclose(g["dq"][0, 0], torch.full((1, 64), 1e3, device="cuda")) and g["dk"] is None


def test_in_place_and_overlap():
    c = make(2, 5, 4, 4, 128, 128, torch.bfloat16, 24)
    kw = dict(cos=c["cos"], sin=c["sin"], pos=c["pos"], mode="rms")
    want = kda.qk_norm_rope(c["q"], c["k"], c["wq"], c["wk"], **kw)
    q, k = c["q"].clone(), c["k"].clone()
    kda.qk_norm_rope(q, k, c["wq"], c["wk"], out=(q, k), **kw)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    with pytest.raises(kda.KDAError):
        kda.qk_norm_rope(q, k, out=(k, q))
    with pytest.raises(ValueError):
        kda.qk_norm_rope(q, k, c["wq"][:64], c["wk"], **kw)
    with pytest.raises(TypeError):
        kda.qk_norm_rope(q, k.float())


def test_sum_norm_is_the_layer_calls_normalisation():
    # the rows kda_fwd_chunked_layer normalises inside: the plain prefill on
    # rows from this call, on the same fp32 gate, gives its result
    from kda_testutil import TOL, err_ratio, f32
    r = np.random.default_rng(25)
    B, T, H = 1, 130, 2
    q, k, v = (cast(2 * r.standard_normal((B, T, H, 128)), torch.bfloat16).cuda() for _ in range(3))
    beta = cast(r.uniform(0, 1, (B, T, H)), torch.bfloat16).cuda()
    z = cast(r.standard_normal((B, T, H, 128)), torch.bfloat16).cuda()
    A = torch.zeros(H, device="cuda")
    g, _ = kda.prepare_decay(z, A, want_gcum=False)
    qn, kn = kda.qk_norm_rope(q, k)
    o, ht = kda.fwd_chunked(qn, kn, v, g, beta)
    o2, ht2 = kda.fwd_chunked_layer(q, k, v, z, A, beta, qk_l2norm=True)
    torch.cuda.synchronize()
    assert err_ratio(f32(o), f32(o2)) <= TOL[torch.bfloat16] and err_ratio(f32(ht), f32(ht2)) <= TOL[torch.bfloat16]


def test_captured_and_replayed():
    c = make(2, 20, 4, 2, 128, 64, torch.bfloat16, 26)
    kw = dict(cos=c["cos"], sin=c["sin"], pos=c["pos"], mode="rms")
    qo, ko = torch.empty_like(c["q"]), torch.empty_like(c["k"])
    out = {"dq": torch.empty_like(qo), "dk": torch.empty_like(ko), "dwq": torch.empty_like(c["wq"]), "dwk": torch.empty_like(c["wk"])}
    ws = torch.empty(kda.lib().kda_qk_bwd_workspace_bytes(2, 20, 4, 2, 128), dtype=torch.uint8, device="cuda")

    def work():
        kda.qk_norm_rope(c["q"], c["k"], c["wq"], c["wk"], out=(qo, ko), **kw)
        kda.qk_norm_rope_bwd(c["q"], c["k"], c["dq"], c["dk"], c["wq"], c["wk"], workspace=ws, out=out, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        work()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        work()
    for _ in range(3):
        c["q"].normal_()
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (qo, ko, *out.values())]
        work()
        torch.cuda.synchronize()
        for a, b in zip(got, (qo, ko, *out.values())):
            assert torch.equal(a, b)


def test_more_tokens_than_one_launch_holds():
    # 70 million tokens of one head: more waves than a launch's 2^32 threads
    T, d = 70_000_003, 8
    say(f"qk norm T={T} Hq=1 d={d}")
    q = torch.randn(1, T, 1, d, device="cuda", dtype=torch.bfloat16)
    whole, _ = kda.qk_norm_rope(q, None, mode="rms")
    for a, b in ((0, 30_000_000), (30_000_000, 60_000_000), (60_000_000, T)):
        part, _ = kda.qk_norm_rope(q[:, a:b], None, mode="rms")
        assert torch.equal(whole[:, a:b], part)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("mode", ["l2", "rms"])
@pytest.mark.parametrize("Hq,Hk,d,rot", [(4, 2, 128, 64), (1, 1, 64, 0), (3, 5, 96, 96), (9, 8, 128, 0), (1, 3, 512, 16)])
def test_weight_gradients_without_an_epsilon(dtype, mode, Hq, Hk, d, rot):
    # eps = 0 on rows that are not zero: lanes that hold no head add nothing to
    # the weights' gradients.  Tolerances as above (no epsilon enters them).
    say(f"qk bwd eps=0 {dtype} {mode} Hq={Hq} Hk={Hk} d={d} rot={rot}")
    B, T, rms = 2, 5, mode == "rms"
    c = make(B, T, Hq, Hk, d, rot, dtype, 27)
    cos, sin = table(c)
    kw = dict(cos=c["cos"], sin=c["sin"], pos=c["pos"], mode=mode, eps=0.0)
    qo, ko = kda.qk_norm_rope(c["q"], c["k"], c["wq"], c["wk"], **kw)
    g = kda.qk_norm_rope_bwd(c["q"], c["k"], c["dq"], c["dk"], c["wq"], c["wk"], **kw)
    torch.cuda.synchronize()
    for n, out, H in (("q", qo, Hq), ("k", ko, Hk)):
        x, w, dy = f64(c[n]).reshape(B * T, H, d), f64(c["w" + n]), f64(c["d" + n]).reshape(B * T, H, d)
        want, size = mix.qk_fwd(x, w, cos, sin, rms, False, 0.0), pair_size(mix.qk_fwd(x, w, None, None, rms, False, 0.0), rot, False)
        check(n, out.reshape(B * T, H, d), want, 18 * U * size, dtype)
        dx, dw = mix.qk_bwd(x, w, cos, sin, dy, rms, False, 0.0)
        r, gs = mix._rinv(x, rms, 0.0), pair_size(dy, rot, False)
        sq = (gs * np.abs(w) * np.abs(x)).sum(-1, keepdims=True) / (d if rms else 1)
        check("dw" + n, g["dw" + n], dw, (25 + 40 + B * T * H / 1024) * U * (gs * np.abs(x) * r).sum((0, 1)), torch.float32)
        check("d" + n, g["d" + n].reshape(B * T, H, d), dx, 30 * U * (gs * np.abs(w) * r + np.abs(x) * r ** 3 * sq), dtype)
