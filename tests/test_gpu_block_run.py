"""The norm of the residual stream, the product of 8-bit rows and the gated
linear recurrence run together, with the short convolution, as a recurrent
block uses them: prompt, tokens behind it, gradients, captured and replayed, on
two streams.

Each stage gets what the stage before it wrote on the GPU and is held to the
fp64 oracle on exactly that (the tolerances of the stage's own tests), so that a
wrong layout, stride or order between two of them shows.
"""
import numpy as np
import pytest
import torch

import test_gpu_conv as tc
import test_gpu_gemm8 as tg
import test_gpu_lru as tl
import test_gpu_rmsnorm as tn
from gated_delta_rule_96_amd import kda
from kda_testutil import cast, say
from oracle import block

pytestmark = pytest.mark.gpu
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
W, EPS = 4, 1e-6


def make(lens, D, E, seed, stream=F32):
    """Residual stream of width D, recurrence of E channels (x, r, i side by side in the projection)."""
    r = np.random.default_rng(seed)
    T, N = sum(lens), len(lens)
    v = lambda a, t=F32: cast(a, t).cuda()
    w = r.standard_normal((3 * E, D)) / np.sqrt(D)
    kb, nb = (D + 127) // 128, (3 * E + 127) // 128
    sw = np.array([[np.abs(w[n * 128:n * 128 + 128, k * 128:k * 128 + 128]).max() / 448 for k in range(kb)] for n in range(nb)]).astype(np.float32)
    w8 = v(w / block.spread(block.spread(sw.astype(np.float64), D), 3 * E, 0)).to(F8)
    return dict(x=v(r.standard_normal((1, T, D)), BF), res=v(2 * r.standard_normal((1, T, D)), stream), w=v(1 + 0.2 * r.standard_normal(D)), w8=w8, sw=v(sw),
                cw=v(r.uniform(-0.7, 0.7, (E, W))), cb=v(r.uniform(-0.5, 0.5, E)), s0=v(r.standard_normal((N, W - 1, E)), BF), c=v(-np.log(r.uniform(0.5, 0.999, E))),
                h0=v(r.standard_normal((N, E))))


def forward(k, cu, E, step=False, s0=None, h0=None):
    """Stages of the block: ((y8, scale), h, projection, convolved x, states, y)."""
    (y8, sc), h = kda.add_rms_norm(k["x"], k["res"], k["w"], eps=EPS, fp8=True)
    p = kda.gemm_fp8(y8, sc, k["w8"], k["sw"])
    x, r, i = p.split(E, -1)
    if step:
        xc = kda.conv_step(x[0], k["cw"], k["cb"], s0)
        y = kda.lru_step(xc, r[0], i[0], k["c"], h0)
        return (y8, sc), h, p, xc[None], s0, y[None], h0
    xc, st = kda.conv_fwd(x, k["cw"], k["cb"], s0, cu_seqlens=cu)
    y, ht = kda.lru_fwd(xc, r, i, k["c"], h0, cu_seqlens=cu)
    return (y8, sc), h, p, xc, st, y, ht


def held(k, lens, E, got, s0, h0):
    """Every stage against its oracle on what it was given."""
    (y8, sc), h, p, xc, st, y, ht = got
    D = k["x"].shape[-1]
    assert torch.equal(h, (k["x"].float() + k["res"].float()).to(h.dtype))
    tn.check8(y8.reshape(-1, D), sc.reshape(-1, sc.shape[-1]), block.rms_norm(tn.f64(h).reshape(-1, D), tn.f64(k["w"]), EPS))
    tg.check(y8.reshape(-1, D), sc.reshape(-1, sc.shape[-1]), k["w8"], k["sw"], p.reshape(-1, 3 * E))
    x, r, i = p[0].split(E, -1)
    yr, sr, ty = tc.oracle_fwd(dict(x=x, w=k["cw"], bias=k["cb"], s0=s0), lens, True)
    tc.check("conv", xc[0], yr, ty, BF)
    assert np.array_equal(tc.f64(st), sr)
    case = dict(x=xc, r=r[None], i=i[None], c=k["c"], h0=h0, dy=None, dht=None)
    want = tl.oracle(case, lens, True)
    tl.check("y", y[0], want["y"], want["ty"], BF)
    tl.check("ht", ht, want["ht"], want["tht"], F32)


@pytest.mark.parametrize("stream", [BF, F32])
@pytest.mark.parametrize("lens,D,E", [([70, 1, 0, 300], 256, 192), ([1100], 400, 128), ([5], 64, 40)])
def test_block_of_prompts_and_the_tokens_behind(lens, D, E, stream):
    say(f"block {lens} D={D} E={E} {stream}")
    k = make(lens, D, E, 7, stream)
    got = forward(k, tl.cuts(lens), E, s0=k["s0"], h0=k["h0"])
    torch.cuda.synchronize()
    held(k, lens, E, got, k["s0"], k["h0"])
    st, state, N = got[4].clone(), got[6].clone(), len(lens)
    for t in range(3):
        more = make([1] * N, D, E, 100 + t, stream)
        one = dict(k, x=more["x"], res=more["res"])
        s0, h0 = st.clone(), state.clone()
        got = forward(one, None, E, step=True, s0=st, h0=state)
        torch.cuda.synchronize()
        held(one, [1] * N, E, got, s0, h0)


def test_gradients_of_a_block():
    # norm in the stream's type, a projection by torch, convolution and recurrence
    lens, D, E = [90, 260], 128, 64
    cu = tl.cuts(lens)
    k = make(lens, D, E, 8)
    r = np.random.default_rng(9)
    T = sum(lens)
    wp = cast(r.standard_normal((3 * E, D)) / np.sqrt(D), F32).cuda()
    x, res = k["x"].float(), k["res"]
    y, h = kda.add_rms_norm(x, res, k["w"], eps=EPS)
    p = y @ wp.t()
    a, rr, ii = p.split(E, -1)
    s0 = k["s0"].float()
    xc, _ = kda.conv_fwd(a, k["cw"], k["cb"], s0, cu_seqlens=cu)
    out, ht = kda.lru_fwd(xc, rr, ii, k["c"], k["h0"], cu_seqlens=cu)
    dout, dht, dh = (cast(r.standard_normal(s), F32).cuda() for s in ((1, T, E), (2, E), (1, T, D)))
    g = kda.lru_bwd(xc, rr, ii, k["c"], dout, k["h0"], dht, cu_seqlens=cu)
    gc = kda.conv_bwd(a, k["cw"], k["cb"], g["dx"], s0, cu_seqlens=cu)
    dp = torch.cat([gc["dx"], g["dr"], g["di"]], -1)
    gn = kda.add_rms_norm_bwd(h, k["w"], dp @ wp, dh, eps=EPS)
    torch.cuda.synchronize()
    case = dict(x=xc, r=rr, i=ii, c=k["c"], h0=k["h0"], dy=dout, dht=dht)
    tl.compare_grads(case, g, tl.oracle(case, lens, True, back=True), F32)
    # The whole chain against differences of the whole chain: central
    # differences with step e are off by e^2 of the third derivative (bounded by
    # 8 S) and by the values' rounding, 400 u S / e, S the sum of the loss's terms.
    loss = lambda hh: _loss(hh, k, wp, s0, cu, E, dout, dht, dh)
    d = cast(r.standard_normal((1, T, D)), F32).cuda()
    S = float((dout.abs() * out.abs()).double().sum() + (dht.abs() * ht.abs()).double().sum() + (dh.abs() * h.abs()).double().sum())
    e = 2.0 ** -7
    slope = (loss(h + e * d) - loss(h - e * d)) / (2 * e)
    assert abs(slope - float((gn["dx"].double() * d.double()).sum())) <= (8 * e * e + 400 * tl.U / e) * S


def _loss(h, k, wp, s0, cu, E, dout, dht, dh):
    y, _ = kda.add_rms_norm(h, None, k["w"], eps=EPS)
    a, r, i = (y @ wp.t()).split(E, -1)
    xc, _ = kda.conv_fwd(a, k["cw"], k["cb"], s0, cu_seqlens=cu)
    out, ht = kda.lru_fwd(xc, r, i, k["c"], k["h0"], cu_seqlens=cu)
    return float((out.double() * dout.double()).sum() + (ht.double() * dht.double()).sum() + (h.double() * dh.double()).sum())


def test_two_graphs_share_workspaces_and_two_streams_do_not():
    # two captured graphs on one workspace, replayed in turn; then the same work
    # on two streams at once, each with its own
    lens, D, E = [700, 64, 300], 256, 192
    cu, T, N = tl.cuts(lens), sum(lens), len(lens)
    L = kda.lib()
    sizes = [L.kda_lru_workspace_bytes(1, T, E, N), L.kda_lru_bwd_workspace_bytes(1, T, E, N), L.kda_add_rms_norm_bwd_workspace_bytes(T, D)]
    space = lambda: [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]

    def worker(seed, ws):
        k = make(lens, D, E, seed)
        r = np.random.default_rng(seed)
        dy, g = cast(r.standard_normal((1, T, E)), BF).cuda(), cast(r.standard_normal((1, T, D)), BF).cuda()
        out = {}

        def work():
            (y8, sc), h = kda.add_rms_norm(k["x"], k["res"], k["w"], eps=EPS, fp8=True)
            x, rr, ii = kda.gemm_fp8(y8, sc, k["w8"], k["sw"]).split(E, -1)
            y, ht = kda.lru_fwd(x, rr, ii, k["c"], k["h0"], cu_seqlens=cu, workspace=ws[0])
            gr = kda.lru_bwd(x, rr, ii, k["c"], dy, k["h0"], ht, cu_seqlens=cu, workspace=ws[1])
            gn = kda.add_rms_norm_bwd(h, k["w"], g, None, eps=EPS, workspace=ws[2])
            out.update(h=h, y=y, ht=ht, dr=gr["dr"], dc=gr["dc"], dh0=gr["dh0"], dx=gn["dx"], dw=gn["dw"])
        return k, out, work
    ws = space()
    sides = [worker(75, ws), worker(76, ws)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _, _, work in sides:
            work()
    torch.cuda.current_stream().wait_stream(s)
    graphs = []
    for _, out, work in sides:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            work()
        graphs.append((g, dict(out)))
    for _ in range(3):
        for k, _, _ in sides:
            k["x"].normal_()
        for w in ws:
            w.fill_(255)
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
    for k, _, _ in own:
        k["x"].normal_()
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


@pytest.mark.parametrize("dtype", [F32, BF])
def test_tokens_far_apart(dtype):
    # token strides of 2^24 elements: offsets behind 2^32 bytes, and behind 2^31 elements
    T, ld, D = 150, 1 << 24, 72
    say(f"token stride 2^24 {dtype}")
    wide = torch.empty((1, T, ld), dtype=dtype, device="cuda")
    near = cast(np.random.default_rng(77).standard_normal((1, T, 3 * D)), dtype).cuda()
    at = ld - 3 * D - 8
    wide[..., at:at + 3 * D].copy_(near)
    c = cast(np.random.default_rng(78).uniform(0.01, 0.5, D), F32).cuda()
    dy = cast(np.random.default_rng(79).standard_normal((1, T, D)), dtype).cuda()

    def run(row):
        x, r, i = row.split(D, -1)
        y, ht = kda.lru_fwd(x, r, i, c)
        g = kda.lru_bwd(x, r, i, c, dy)
        yt = kda.lru_step(x[0], r[0], i[0], c, torch.ones((T, D), device="cuda"))
        n, h = kda.add_rms_norm(x, r)
        gn = kda.add_rms_norm_bwd(x, None, dy, want_dw=True)
        torch.cuda.synchronize()
        return [y, ht, yt, n, h, gn["dx"], gn["dw"]] + [t for t in g.values() if t is not None]
    for a, b in zip(run(wide[..., at:at + 3 * D]), run(near)):
        assert torch.isfinite(a).all() and torch.equal(a, b)


def test_long_cache_of_rows():
    # more than 2^32 elements in one call: rows behind them are computed like the first
    R, D = (1 << 32) // 4096 + 70, 4096
    x = torch.empty((R, D), dtype=BF, device="cuda")
    x[:64].normal_()
    x[64:128].copy_(x[:64])
    x[-64:].copy_(x[:64])
    x[128:-64].zero_()
    (y8, sc), _ = kda.add_rms_norm(x, fp8=True)
    g = kda.add_rms_norm_bwd(x, None, x)
    torch.cuda.synchronize()
    assert torch.equal(y8[-64:].view(torch.uint8), y8[:64].view(torch.uint8)) and torch.equal(sc[-64:], sc[:64]) and torch.equal(g["dx"][-64:], g["dx"][:64])
    w8 = torch.zeros((8, D), device="cuda").to(F8)
    w8[:, :8] = torch.eye(8, device="cuda").to(F8)
    c = kda.gemm_fp8(y8, sc, w8, torch.ones((1, 32), device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(c[-64:], c[:64]) and torch.equal(c[64:128], c[:64])
    # the recurrence over the same rows as one sequence, and over its end alone:
    # cut at a multiple of the 128 tokens of a part, so that the sums' order is
    # the same (a token's place in its part decides where partial sums round)
    del y8, sc, c
    L = 2048 + R % 128
    y, ht = kda.lru_fwd(x.view(1, R, D), x.view(1, R, D), None, torch.ones(D, device="cuda"), final_state=True, unit=False)
    tail, _ = kda.lru_fwd(x[-L:].view(1, L, D), x[-L:].view(1, L, D), None, torch.ones(D, device="cuda"), unit=False)
    torch.cuda.synchronize()
    # 2000 tokens of decay e^-1/2 and more forget everything before them
    assert torch.equal(y[0, -64:], tail[0, -64:])


def test_more_work_than_the_usual_tiles_have_groups_for():
    # the product: more outputs of one row than work-groups of 16 or 64 outputs,
    # more rows than tiles of 64; the norm: more rows than one work-group each
    one = torch.ones((1, 1), device="cuda")
    N = (1 << 27) + 200
    say(f"product 1 x {N} x 16")
    w8 = torch.empty((N, 16), dtype=torch.uint8, device="cuda").fill_(56).view(F8)
    w8[:300] = torch.randn((300, 16), device="cuda").to(F8)
    w8[-300:] = torch.randn((300, 16), device="cuda").to(F8)
    a8 = torch.randn((1, 16), device="cuda").to(F8)
    sw = torch.rand(((N + 127) // 128, 1), device="cuda")
    c = kda.gemm_fp8(a8, one, w8, sw)
    cut = N // 128 * 128 - 128
    assert torch.equal(c[:, cut:], kda.gemm_fp8(a8, one, w8[cut:], sw[cut // 128:])) and torch.equal(c[:, :256], kda.gemm_fp8(a8, one, w8[:256], sw[:2]))
    del w8, c
    M = (1 << 29) + 700
    say(f"product {M} x 8 x 16")
    a8 = torch.empty((M, 16), dtype=torch.uint8, device="cuda").fill_(56).view(F8)
    a8[-900:] = torch.randn((900, 16), device="cuda").to(F8)
    sa, w8 = torch.ones((M, 1), device="cuda"), torch.randn((8, 16), device="cuda").to(F8)
    sa[-900:].uniform_()
    c = kda.gemm_fp8(a8, sa, w8, one)
    assert torch.equal(c[-900:], kda.gemm_fp8(a8[-900:], sa[-900:], w8, one)) and torch.equal(c[:900], kda.gemm_fp8(a8[:900], sa[:900], w8, one))
    del a8, sa, c
    R = (1 << 22) + 77
    say(f"norm {R} x 8")
    x = torch.randn((R, 8), dtype=BF, device="cuda")
    y, _ = kda.add_rms_norm(x)
    assert torch.equal(y[-900:], kda.add_rms_norm(x[-900:].contiguous())[0])


def test_chains_of_parts_beside_other_work():
    # two long recurrences (one that looks back near, one far) and products on
    # streams of their own, all at once: the same bits as one after the other
    r = np.random.default_rng(81)
    t = lambda *s: cast(r.standard_normal(s), BF).cuda()
    a, b = [t(1, 30000, 1400) for _ in range(3)], [t(1, 60000, 64) for _ in range(3)]
    ca, cb = (cast(-np.log(r.uniform(0.9, 0.999, n)), F32).cuda() for n in (1400, 64))
    m8, w8 = (torch.randn((n, 2048), device="cuda").to(F8) for n in (3000, 2500))
    sa, sw = torch.rand((3000, 16), device="cuda"), torch.rand((20, 16), device="cuda")
    jobs = [lambda: kda.lru_fwd(*a, ca)[0], lambda: kda.lru_fwd(*b, cb)[0], lambda: kda.gemm_fp8(m8, sa, w8, sw), lambda: kda.lru_bwd(*b, cb, b[0])["dr"]]
    want = [j() for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [[] for _ in jobs]
    for _ in range(6):
        for j, s, g in zip(jobs, streams, got):
            with torch.cuda.stream(s):
                g.append(j())
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(w, o) for o in g)
