"""The convolution, the head norms and the scan run together with the gated
delta rule, as a layer uses them: prompt, gradients, tokens behind the prompt.

Each stage gets what the stage before it wrote on the GPU and is held to the
fp64 oracle on exactly that (the tolerances of the stage's own tests), so that
a wrong layout, stride or order between two of them shows.  Whole chains are
held to the chain of oracles: their tolerances stand at the tests.
"""
import numpy as np
import pytest
import torch

import test_gpu_conv as tc
import test_gpu_qknorm as tq
import test_gpu_ssm as ts
import test_gpu_ssm_bwd as tb
from gated_delta_rule_96_amd import kda, synth
from kda_testutil import TOL, cast, err_ratio, f32, say
from oracle import mix, seq
from test_gpu_bwd import grad_err

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DTYPES = [torch.float32, torch.bfloat16]
W, D1, ROT = 4, 128, 64


def angles(n):
    a = np.arange(n)[:, None] * 10000.0 ** (-np.arange(0, ROT, 2) / ROT)
    return cast(np.cos(a), torch.float32).cuda(), cast(np.sin(a), torch.float32).cuda()


def block(B, T, H, dtype, seed):
    """Inputs of a block: projections of q, k, v side by side, gates, states."""
    r = np.random.default_rng(seed)
    D = 3 * H * D1
    v = lambda a, t=torch.float32: cast(a, t).cuda()
    return dict(x=v(r.standard_normal((B, T, D)), dtype), w=v(r.uniform(-0.7, 0.7, (D, W))), bias=v(r.uniform(-0.5, 0.5, D)),
                s0=v(r.standard_normal((B, W - 1, D)), dtype), g=v(-r.uniform(0.01, 1.0, (B, T, H, D1)), dtype),
                beta=v(r.uniform(0.1, 0.9, (B, T, H)), dtype), h0=v(0.3 * r.standard_normal((B, H, D1, D1))),
                do=v(r.standard_normal((B, T, H, D1))), dht=v(r.standard_normal((B, H, D1, D1))))


def heads(y, H):
    """q, k and v heads of a convolved row: slices."""
    return [t.unflatten(-1, (H, D1)) for t in y.split(H * D1, -1)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,T,H", [(2, 130, 2), (1, 64, 1), (3, 1, 2)])
def test_linear_attention_block_and_its_gradients(dtype, B, T, H):
    say(f"block {dtype} B={B} T={T} H={H}")
    c = block(B, T, H, dtype, 71)
    cos, sin = angles(T + 7)
    rope = dict(cos=cos, sin=sin, pos0=7, mode="l2")
    y, st = kda.conv_fwd(c["x"], c["w"], c["bias"], c["s0"])
    q, k, v = heads(y, H)
    qn, kn = kda.qk_norm_rope(q, k, **rope)
    v = v.contiguous()
    o, ht = kda.fwd_chunked(qn, kn, v, c["g"], c["beta"], c["h0"])
    g = kda.bwd_chunked(qn, kn, v, c["g"], c["beta"], c["h0"], c["do"], c["dht"])
    gq = kda.qk_norm_rope_bwd(q, k, g["dq"], g["dk"], **rope)
    dy = torch.cat([gq["dq"].float().flatten(2), gq["dk"].float().flatten(2), g["dv"].flatten(2)], -1)
    gx = kda.conv_bwd(c["x"], c["w"], c["bias"], dy, c["s0"])
    torch.cuda.synchronize()

    # stage by stage
    lens = [T] * B
    flat = dict(x=c["x"].flatten(0, 1), w=c["w"], bias=c["bias"], s0=c["s0"], dy=dy.flatten(0, 1))
    yr, sr, ty = tc.oracle_fwd(flat, lens, True)
    tc.check("conv", y.flatten(0, 1), yr, ty, dtype)
    assert np.array_equal(tc.f64(st), sr)
    cc, ss = (np.tile(f32(t).astype(np.float64)[7:7 + T], (B, 1)) for t in (cos, sin))
    for n, x, out, up, dx in (("q", q, qn, g["dq"], gq["dq"]), ("k", k, kn, g["dk"], gq["dk"])):
        x, up = tc.f64(x).reshape(B * T, H, D1), tc.f64(up).reshape(B * T, H, D1)
        want = mix.qk_fwd(x, None, cc, ss, False, False)
        tq.check(n, out.reshape(B * T, H, D1), want, 18 * U * tq.pair_size(mix.qk_fwd(x, None, None, None, False, False), ROT, False), dtype)
        dref, _ = mix.qk_bwd(x, None, cc, ss, up, False, False)
        r, gs = mix._rinv(x, False, 1e-6), tq.pair_size(up, ROT, False)
        tq.check("d" + n, dx.reshape(B * T, H, D1), dref, 30 * U * (gs * r + np.abs(x) * r ** 3 * (gs * np.abs(x)).sum(-1, keepdims=True)), dtype)
    args = [f32(t) for t in (qn, kn, v, c["g"], c["beta"], c["h0"])]
    oref, href = seq.kda_seq(*args)
    assert err_ratio(f32(o), oref) <= TOL[dtype] and err_ratio(f32(ht), href) <= TOL[dtype]
    gref = seq.kda_seq_bwd(*args, f32(c["do"]), f32(c["dht"]))
    for n in ("dq", "dk", "dv", "dg", "dbeta", "dh0"):
        assert grad_err(f32(g[n]), gref[n]) <= TOL[dtype], n
    want, tol = tc.grads_case(flat, lens, True, False)
    for n, x, ref, t in zip(("dx", "dw", "dbias", "ds0"), (gx["dx"].flatten(0, 1), gx["dw"], gx["dbias"], gx["ds0"]), want, tol):
        tc.check(n, x, ref, t, dtype if n in ("dx", "ds0") else torch.float32)

    # The whole chain in fp32 against the chain of oracles.  The gated delta
    # rule's gradients are off by 1e-4 (rms + |ref|); the norm's projection
    # passes at most twice that, the convolution W |w| |act'| <= 4 x 0.7 x 1.1
    # of it, and their own errors are below 1e-5: 1e-3 in all.
    if dtype == torch.float32:
        qr, kr, vr = (a.reshape(B, T, H, D1) for a in np.split(yr.reshape(B, T, -1), 3, -1))
        turn = lambda a: mix.qk_fwd(a.reshape(B * T, H, D1), None, cc, ss, False, False).reshape(B, T, H, D1)
        gref = seq.kda_seq_bwd(*(a.astype(np.float32) for a in (turn(qr), turn(kr), vr)), *args[3:], f32(c["do"]), f32(c["dht"]))
        back = lambda a, up: mix.qk_bwd(a.reshape(B * T, H, D1), None, cc, ss, np.asarray(up, np.float64).reshape(B * T, H, D1), False, False)[0]
        dyr = np.concatenate([back(qr, gref["dq"]).reshape(B, T, -1), back(kr, gref["dk"]).reshape(B, T, -1),
                              np.asarray(gref["dv"], np.float64).reshape(B, T, -1)], -1)
        for i in range(B):
            ref = mix.conv_bwd(tc.f64(c["x"])[i], tc.f64(c["w"]), tc.f64(c["bias"]), tc.f64(c["s0"])[i], dyr[i], None, True)
            assert grad_err(f32(gx["dx"])[i], ref[0]) <= 1e-3 and grad_err(f32(gx["ds0"])[i], ref[3]) <= 1e-3


@pytest.mark.parametrize("dtype", DTYPES)
def test_linear_attention_tokens_behind_the_prompt(dtype):
    # a prompt of 97 tokens and 6 single tokens against the oracles over all 103
    # at once: two roundings of the inputs apart at most (TOL each)
    B, T, n, H = 3, 97, 6, 2
    say(f"prompt and tokens {dtype}")
    c = block(B, T + n, H, dtype, 72)
    cos, sin = angles(T + n)
    cut = lambda t: t[:, :T].contiguous()
    y, st = kda.conv_fwd(cut(c["x"]), c["w"], c["bias"], c["s0"])
    q, k, v = heads(y, H)
    qn, kn = kda.qk_norm_rope(q, k, cos=cos, sin=sin)
    o, state = kda.fwd_chunked(qn, kn, v.contiguous(), cut(c["g"]), cut(c["beta"]), c["h0"])
    got = []
    for t in range(T, T + n):
        yt = kda.conv_step(c["x"][:, t], c["w"], c["bias"], st)
        q, k, v = (a[:, None] for a in heads(yt, H))
        pos = torch.full((B, 1), t, dtype=torch.int32, device="cuda")
        qn, kn = kda.qk_norm_rope(q, k, cos=cos, sin=sin, pos=pos)
        got.append(kda.decode_step(qn[:, 0], kn[:, 0], v[:, 0].contiguous(), c["g"][:, t].contiguous(), c["beta"][:, t].contiguous(), state))
    torch.cuda.synchronize()
    lens = [T + n] * B
    yr, sr, _ = tc.oracle_fwd(dict(x=c["x"].flatten(0, 1), w=c["w"], bias=c["bias"], s0=c["s0"]), lens, True)
    rnd = lambda a: cast(a, dtype).double().numpy()
    qr, kr, vr = (a.reshape(B, T + n, H, D1) for a in np.split(rnd(yr).reshape(B, T + n, -1), 3, -1))
    cc, ss = (np.tile(f32(t).astype(np.float64), (B, 1)) for t in (cos, sin))
    turn = lambda a: rnd(mix.qk_fwd(a.reshape(-1, H, D1), None, cc, ss, False, False)).reshape(B, T + n, H, D1)
    oref, href = seq.kda_seq(*(a.astype(np.float32) for a in (turn(qr), turn(kr), vr)), f32(c["g"]), f32(c["beta"]), f32(c["h0"]))
    assert err_ratio(f32(o), oref[:, :T]) <= 2 * TOL[dtype]
    assert err_ratio(np.stack([f32(t) for t in got], 1), oref[:, T:]) <= 2 * TOL[dtype]
    assert err_ratio(f32(state), href) <= 2 * TOL[dtype]
    assert np.array_equal(tc.f64(st), sr)


def scan_block(lens, H, G, dk, dv, dtype, seed):
    """A projection row: x, B, C (through the convolution), then step sizes."""
    r = np.random.default_rng(seed)
    T, N, D = sum(lens), len(lens), H * dv + 2 * G * dk
    row = cast(r.standard_normal((1, T, D + (H + 7) // 8 * 8)), dtype).cuda()
    v = lambda a, t=torch.float32: cast(a, t).cuda()
    return dict(row=row, D=D, w=v(r.uniform(-0.7, 0.7, (D, W))), cb=v(r.uniform(-0.5, 0.5, D)), s0=v(r.standard_normal((N, W - 1, D)), dtype),
                A=v(-r.uniform(1, 8, H)), bias=v(r.uniform(-4, -2, H)), skip=v(r.standard_normal(H)), h0=v(0.5 * r.standard_normal((N, H, dk, dv))))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens,H,G,dk,dv", [([70, 1, 0, 130], 4, 2, 128, 64), ([700], 2, 1, 128, 128), ([5, 3], 3, 1, 64, 64)])
def test_scan_block_its_tokens_and_its_gradients(dtype, lens, H, G, dk, dv):
    say(f"scan block {dtype} {lens} H={H} G={G}")
    c = scan_block(lens, H, G, dk, dv, dtype, 73)
    N, T, D, cu = len(lens), sum(lens), c["D"], tc.cuts(lens)
    widths = [H * dv, G * dk, G * dk]

    def parts(y):
        a, b, d = y.split(widths, -1)
        return a.unflatten(-1, (H, dv)), b.unflatten(-1, (G, dk)), d.unflatten(-1, (G, dk))
    x, raw = c["row"][..., :D], c["row"][..., D:D + H]
    y, st = kda.conv_fwd(x, c["w"], c["cb"], c["s0"], cu_seqlens=cu)
    xs, Bm, Cm = parts(y)
    kw = dict(D=c["skip"], dt_bias=c["bias"], softplus=True)
    o, ht = kda.ssm_fwd_chunked(xs, raw, c["A"], Bm, Cm, c["h0"], cu_seqlens=cu, **kw)
    r = np.random.default_rng(74)
    do, dht = cast(r.standard_normal((1, T, H, dv)), dtype).cuda(), cast(r.standard_normal((N, H, dk, dv)), torch.float32).cuda()
    g = kda.ssm_bwd_chunked(xs, raw, c["A"], Bm, Cm, do, c["h0"], dht, cu_seqlens=cu, **kw)
    dy = torch.cat([g["dx"].flatten(2), g["dB"].flatten(2), g["dC"].flatten(2)], -1)
    gx = kda.conv_bwd(x, c["w"], c["cb"], dy, c["s0"], cu_seqlens=cu)
    torch.cuda.synchronize()
    flat = dict(x=x[0], w=c["w"], bias=c["cb"], s0=c["s0"], dy=dy[0])
    yr, sr, ty = tc.oracle_fwd(flat, lens, True)
    tc.check("conv", y[0], yr, ty, dtype)
    assert np.array_equal(tc.f64(st), sr)
    case = dict(x=xs[0], dt=raw[0], A=c["A"], B=Bm[0], C=Cm[0], h0=c["h0"], D=c["skip"], bias=c["bias"], soft=True, dy=do[0], dht=dht)
    want = ts.oracle(case, lens, dtype)
    ts.check("y", o[0], want[0], want[2], dtype)
    ts.check("ht", ht, want[1], want[3], torch.float32)
    tb.compare(case, g, tb.oracle(case, lens), lens, dtype)
    want, tol = tc.grads_case(flat, lens, True, False)
    for n, a, ref, t in zip(("dx", "dw", "dbias", "ds0"), (gx["dx"][0], gx["dw"], gx["dbias"], gx["ds0"]), want, tol):
        tc.check(n, a, ref, t, dtype if n in ("dx", "ds0") else torch.float32)

    # three more tokens of every sequence, states moved on in place
    more = cast(r.standard_normal((N, 3, c["row"].shape[-1])), dtype).cuda()
    state = ht.clone()
    for t in range(3):
        before, sb = state.clone(), st.clone()
        yt = kda.conv_step(more[:, t, :D], c["w"], c["cb"], st)
        a, b, d = parts(yt)
        ot = kda.ssm_step(a, more[:, t, D:D + H], c["A"], b, d, state, **kw)
        torch.cuda.synchronize()
        one = [1] * N
        yr, sr, ty = tc.oracle_fwd(dict(x=more[:, t, :D], w=c["w"], bias=c["cb"], s0=sb), one, True)
        tc.check("conv step", yt, yr, ty, dtype)
        assert np.array_equal(tc.f64(st), sr)
        case = dict(x=a, dt=more[:, t, D:D + H], A=c["A"], B=b, C=d, h0=before, D=c["skip"], bias=c["bias"], soft=True)
        want = ts.oracle(case, one, dtype)
        ts.check("y step", ot, want[0], want[2], dtype)
        ts.check("state", state, want[1], want[3], torch.float32)


def test_two_graphs_share_workspaces_and_two_streams_do_not():
    # two captured graphs on one workspace, replayed in turn; then the same work
    # on two streams at once, each with its own
    lens, H, dk, dv = [700, 64, 300], 2, 128, 128
    cu, T = tc.cuts(lens), sum(lens)
    L = kda.lib()
    dev = dict(dtype=torch.uint8, device="cuda")
    nf, nb = L.kda_ssm_workspace_bytes(1, T, H, dk, dv, 1), L.kda_ssm_bwd_workspace_bytes(1, T, H, 1, dk, dv, 1, len(lens))
    D = H * dv + 2 * dk
    nc = L.kda_conv_bwd_workspace_bytes(1, T, D, W, len(lens))

    def worker(seed, ws):
        c = scan_block(lens, H, 1, dk, dv, torch.bfloat16, seed)
        x, raw = c["row"][..., :D], c["row"][..., D:D + H]
        do = cast(np.random.default_rng(seed).standard_normal((1, T, H, dv)), torch.bfloat16).cuda()
        kw = dict(D=c["skip"], dt_bias=c["bias"], softplus=True, cu_seqlens=cu)
        out = {}

        def work():
            y, st = kda.conv_fwd(x, c["w"], c["cb"], c["s0"], cu_seqlens=cu)
            a, b, d = y.split([H * dv, dk, dk], -1)
            a, b, d = a.unflatten(-1, (H, dv)), b.unflatten(-1, (1, dk)), d.unflatten(-1, (1, dk))
            o, ht = kda.ssm_fwd_chunked(a, raw, c["A"], b, d, c["h0"], workspace=ws[0], **kw)
            g = kda.ssm_bwd_chunked(a, raw, c["A"], b, d, do, c["h0"], None, workspace=ws[1], **kw)
            dy = torch.cat([g["dx"].flatten(2), g["dB"].flatten(2), g["dC"].flatten(2)], -1)
            gx = kda.conv_bwd(x, c["w"], c["cb"], dy, c["s0"], cu_seqlens=cu, workspace=ws[2])
            out.update(o=o, ht=ht, st=st, ddt=g["ddt"], dA=g["dA"], dh0=g["dh0"], dx=gx["dx"], dw=gx["dw"])
        return c, out, work
    space = lambda: [torch.empty(n, **dev) for n in (nf, nb, nc)]
    ws = space()
    sides = [worker(75, ws), worker(76, ws)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _, _, work in sides:
            work()
    torch.cuda.current_stream().wait_stream(s)
    graphs = []
    for c, out, work in sides:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            work()
        graphs.append((g, dict(out)))
    for _ in range(3):
        for c, _, _ in sides:
            c["row"].normal_()
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        got = [{n: t.clone() for n, t in o.items()} for _, o in graphs]
        for (_, out, work), w in zip(sides, got):
            work()
            torch.cuda.synchronize()
            for n in w:
                assert torch.equal(w[n], out[n]), n
    own = [worker(75, space()), worker(76, space())]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for c, _, _ in own:
        c["row"].normal_()
    torch.cuda.synchronize()
    for _ in range(3):
        for st, (_, _, work) in zip(streams, own):
            with torch.cuda.stream(st):
                work()
        torch.cuda.synchronize()
        got = [{n: t.clone() for n, t in o.items()} for _, o, _ in own]
        for (_, out, work), w in zip(own, got):
            work()
            torch.cuda.synchronize()
            for n in w:
                assert torch.equal(w[n], out[n]), n


@pytest.mark.parametrize("dtype", DTYPES)
def test_tokens_far_apart(dtype):
    # token strides of 2^24 elements: offsets behind 2^32 bytes, and behind 2^31
    # elements, at sizes that a card's memory holds
    T, ld, H, dk, dv = 150, 1 << 24, 2, 64, 64
    say(f"token stride 2^24 {dtype}: {T * ld * dtype.itemsize / 2 ** 30:.1f} GiB")
    wide = torch.empty((1, T, ld), dtype=dtype, device="cuda")
    D = H * dv + 2 * dk
    at = ld - D - 8
    near = cast(np.random.default_rng(77).standard_normal((1, T, D + 8)), dtype).cuda()
    wide[..., at:].copy_(near)
    v = lambda a: cast(a, torch.float32).cuda()
    r = np.random.default_rng(78)
    w, bias, A = v(r.uniform(-0.7, 0.7, (D, W))), v(r.uniform(-0.5, 0.5, D)), v(-r.uniform(1, 4, H))
    do = cast(r.standard_normal((1, T, H, dv)), dtype).cuda()
    dy = cast(r.standard_normal((1, T, D)), dtype).cuda()

    def run(row):
        p = row.split([H * dv, dk, dk, 8], -1)
        x, b, c = p[0].unflatten(-1, (H, dv)), p[1].unflatten(-1, (1, dk)), p[2].unflatten(-1, (1, dk))
        raw = p[3][..., :H]
        y, st = kda.conv_fwd(row[..., :D], w, bias)
        gx = kda.conv_bwd(row[..., :D], w, bias, dy)
        qn, kn = kda.qk_norm_rope(x, b)
        gq = kda.qk_norm_rope_bwd(x, b, do, dy[..., :dk].unflatten(-1, (1, dk)).contiguous())
        o, ht = kda.ssm_fwd_chunked(x, raw, A, b, c, softplus=True)
        g = kda.ssm_bwd_chunked(x, raw, A, b, c, do, softplus=True)
        yt = kda.conv_step(row[0, :, :D], w, bias, torch.zeros((T, W - 1, D), dtype=dtype, device="cuda"))
        ot = kda.ssm_step(x[0], raw[0], A, b[0], c[0], torch.ones((T, H, dk, dv), device="cuda"), softplus=True)
        torch.cuda.synchronize()
        return [y, st, qn, kn, o, ht, yt, ot] + [t for d in (gx, gq, g) for t in d.values() if t is not None]
    for a, b in zip(run(wide[..., at:]), run(near)):
        assert torch.isfinite(a).all() and torch.equal(a, b)
