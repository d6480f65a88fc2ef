"""GPU parity of the short causal convolution (kda_conv_fwd, kda_conv_step,
kda_conv_bwd) against the fp64 oracle (oracle/mix.py) on the cast inputs.

Tolerances, per element.  u = 2^-24, h = half a step of the output type,
finfo.eps / 2 relative to the value.  The sum of W products and the bias is at most W + 1
roundings of partial sums below M = |bias| + sum |w x|: |dz_err| <= (W+1) u M.
Sigmoid through 2^(-z log2 e): relative error (|z| + 4) u.  |act'| <= 1.1,
|act''| <= 0.5.  With the product z Sigmoid(z): |y_err| <= 1.1 (W+1) u M +
(|z| + 6) u |y|, then h |y| for the output's rounding.  dz = dy act'(z): the
error of act' is at most 0.5 (W+1) u M + (2 |z| + 10) u (1 + |z|).  dx and ds0
sum W such dz and a final state's gradient.  dw and dbias add their terms over
at most 64 tokens in a thread, 6 lane steps, 4 waves, then every 16th partial
row and 16 of those: with R rows of tokens at most 90 + R/256 additions, each
off by u times the sum of the terms' sizes, on top of the terms' own errors.
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


def make(lens, D, W, dtype, seed, bias=True, state=True, pad=0):
    """Tokens of all sequences [T,D] as a slice of a tensor `pad` wider."""
    r = np.random.default_rng(seed)
    T, N = sum(lens), len(lens)
    wide = cast(r.standard_normal((T, D + pad)), dtype).cuda()
    return dict(x=wide[:, :D], w=cast(r.uniform(-0.7, 0.7, (D, W)), torch.float32).cuda(),
                bias=cast(r.uniform(-0.5, 0.5, D), torch.float32).cuda() if bias else None,
                s0=cast(r.standard_normal((N, W - 1, D)), dtype).cuda() if state else None,
                dst=cast(r.standard_normal((N, W - 1, D)), dtype).cuda(), dy=cast(r.standard_normal((T, D)), dtype).cuda())


def cuts(lens):
    return np.concatenate([[0], np.cumsum(lens)]).tolist()


def oracle_fwd(c, lens, silu):
    cu, w, b = cuts(lens), f64(c["w"]), f64(c["bias"])
    W = w.shape[1]
    ys, sts, tol = [], [], []
    for i in range(len(lens)):
        y, st, z, rows = mix.conv_fwd(f64(c["x"])[cu[i]:cu[i + 1]], w, b, None if c["s0"] is None else f64(c["s0"])[i], silu)
        n = lens[i]
        M = sum(np.abs(rows[j:j + n] * w[:, j]) for j in range(W)) + (0 if b is None else np.abs(b))
        ys.append(y)
        sts.append(st)
        tol.append(1.1 * (W + 1) * U * M + (np.abs(z) + 6) * U * np.abs(y))
    return np.concatenate(ys), np.stack(sts), np.concatenate(tol)


def check(name, got, want, tol, dtype):
    h = torch.finfo(dtype).eps / 2
    bad = np.abs(f64(got) - want) > tol * (1 + h) + h * np.abs(want)
    worst = float(np.max(np.abs(f64(got) - want) / (tol * (1 + h) + h * np.abs(want) + 1e-300))) if want.size else 0.0
    assert not bad.any(), (name, int(bad.sum()), worst, np.argwhere(bad)[:3].tolist())


# sequence lengths around the window, the strips and the 128 sequences of a launch
LENS = [[1], [2], [3], [7], [64, 64], [200], [5, 0, 1, 130, 0], [3, 1, 1, 2], [0, 4], [1] * 5, [2, 0, 3] * 50, [1] * 257]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens", LENS, ids=lambda l: f"{len(l)}x{sum(l)}")
@pytest.mark.parametrize("D,W,pad,bias,state,silu", [(8, 4, 0, True, True, True), (64, 3, 8, False, True, True), (37, 4, 5, True, False, False),
                                                     (3, 2, 0, True, True, True), (520, 4, 0, True, True, True)])
def test_conv_packed(dtype, lens, D, W, pad, bias, state, silu):
    say(f"conv packed {dtype} N={len(lens)} T={sum(lens)} D={D} W={W} pad={pad}")
    c = make(lens, D, W, dtype, 7, bias, state, pad)
    y_ref, st_ref, tol = oracle_fwd(c, lens, silu)
    y, st = kda.conv_fwd(c["x"][None], c["w"], c["bias"], c["s0"], silu=silu, cu_seqlens=cuts(lens))
    torch.cuda.synchronize()
    check("y", y[0], y_ref, tol, dtype)
    assert np.array_equal(f64(st), st_ref)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,T,D,W", [(1, 1, 64, 4), (3, 2, 40, 4), (2, 300, 128, 3), (5, 65, 13, 2), (2, 1500, 2048, 4)])
def test_conv_batch_and_in_place_state(dtype, B, T, D, W):
    say(f"conv batch {dtype} B={B} T={T} D={D} W={W}")
    c = make([T] * B, D, W, dtype, 8)
    y_ref, st_ref, tol = oracle_fwd(c, [T] * B, True)
    x = c["x"].view(B, T, D)
    s0 = c["s0"].clone()
    y, st = kda.conv_fwd(x, c["w"], c["bias"], s0, st=s0)     # the state replaced in place
    y2, none = kda.conv_fwd(x, c["w"], c["bias"], c["s0"], final_state=False)
    torch.cuda.synchronize()
    assert none is None and st.data_ptr() == s0.data_ptr()
    check("y", y.view(-1, D), y_ref, tol, dtype)
    assert torch.equal(y, y2) and np.array_equal(f64(s0), st_ref)


def test_conv_batch_of_strided_slices():
    # a batch whose tokens are slices of wider rows, at an odd channel offset
    B, T, D = 2, 50, 24
    wide = torch.randn(B, T, 70, device="cuda").to(torch.bfloat16)
    w = torch.randn(D, 4, device="cuda")
    for off in (0, 8, 5):
        x = wide[:, :, off:off + D]
        y, st = kda.conv_fwd(x, w)
        y2, st2 = kda.conv_fwd(x.contiguous(), w)
        assert torch.equal(y, y2) and torch.equal(st, st2)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,D,W,pad", [(1, 8, 4, 0), (5, 37, 3, 1), (300, 64, 2, 8), (7, 4352, 4, 0)])
def test_conv_step_continues_the_prompt(dtype, B, D, W, pad):
    say(f"conv step {dtype} B={B} D={D} W={W}")
    T = 6
    c = make([T] * B, D, W, dtype, 9, pad=pad)
    y_ref, st_ref, tol = oracle_fwd(c, [T] * B, True)
    x = torch.as_strided(c["x"], (B, T, D), (T * (D + pad), D + pad, 1))
    state, ys = c["s0"].clone(), []
    for t in range(T):
        kept = state.clone()
        nxt = torch.full_like(state, float("nan"))
        ya = kda.conv_step(x[:, t], c["w"], c["bias"], state, state_out=nxt)   # the old state stays
        assert torch.equal(state, kept)
        yb = kda.conv_step(x[:, t], c["w"], c["bias"], state)                  # in place
        assert torch.equal(ya, yb) and torch.equal(nxt, state)
        ys.append(ya)
    check("y", torch.stack(ys, 1).view(-1, D), y_ref, tol, dtype)
    assert np.array_equal(f64(state), st_ref)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,D,pad", [(64, 4352, 0), (255, 2061, 3), (257, 4352, 4128), (601, 3999, 1), (1, 40000, 0)])
def test_conv_step_is_a_prompt_of_one_token(dtype, B, D, pad):
    # from few channels and sequences to as many as a thread takes four sequences for
    say(f"conv step {dtype} B={B} D={D} pad={pad}")
    torch.manual_seed(18)
    x = torch.randn(B, D + pad, device="cuda").to(dtype)[:, :D]
    w, bias, state = torch.randn(D, 4, device="cuda"), torch.randn(D, device="cuda"), torch.randn(B, 3, D, device="cuda").to(dtype)
    y, st = kda.conv_fwd(x[:, None], w, bias, state)
    nxt = torch.full_like(state, float("nan"))
    kept = state.clone()
    got = kda.conv_step(x, w, bias, state, state_out=nxt)
    assert torch.equal(got, y[:, 0]) and torch.equal(nxt, st) and torch.equal(state, kept)
    again = kda.conv_step(x, w, bias, state)
    assert torch.equal(again, got) and torch.equal(state, st)


def grads_case(c, lens, silu, dst):
    cu, w, b = cuts(lens), f64(c["w"]), f64(c["bias"])
    W = w.shape[1]
    dxs, ds0s, tx, ts, tw, tb, dw, db = [], [], [], [], 0.0, 0.0, 0.0, 0.0
    for i, n in enumerate(lens):
        s0 = None if c["s0"] is None else f64(c["s0"])[i]
        x, dy = f64(c["x"])[cu[i]:cu[i + 1]], f64(c["dy"])[cu[i]:cu[i + 1]]
        d = f64(c["dst"])[i] if dst else None
        dx, dwi, dbi, ds0, dz = mix.conv_bwd(x, w, b, s0, dy, d, silu)
        _, _, z, rows = mix.conv_fwd(x, w, b, s0, silu)
        M = sum(np.abs(rows[j:j + n] * w[:, j]) for j in range(W)) + (0 if b is None else np.abs(b))
        e = np.abs(dy) * (0.5 * (W + 1) * U * M + (2 * np.abs(z) + 10) * U * (1 + np.abs(z))) if silu else 0 * dz
        t = np.zeros_like(rows)
        size = np.zeros_like(rows)
        for j in range(W):
            t[j:j + n] += e * np.abs(w[:, j])
            size[j:j + n] += np.abs(dz * w[:, j])
        if dst:
            size[n:] += np.abs(d)
        t += (W + 1) * U * size
        dxs.append(dx)
        ds0s.append(ds0)
        tx.append(t[W - 1:])
        ts.append(t[:W - 1])
        dw, db = dw + dwi, db + dbi
        tw = tw + np.stack([(e * np.abs(rows[j:j + n])).sum(0) + (90 + n / 256) * U * np.abs(dz * rows[j:j + n]).sum(0) for j in range(W)], 1)
        tb = tb + e.sum(0) + (90 + n / 256) * U * np.abs(dz).sum(0)
    return (np.concatenate(dxs), dw, db, np.stack(ds0s)), (np.concatenate(tx), tw, tb, np.stack(ts))


@pytest.mark.parametrize("dtype,gtype", [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("lens", [[1], [2], [4], [130], [64, 64, 64], [5, 0, 1, 70, 0, 2], [1] * 140, [0, 300]], ids=lambda l: f"{len(l)}x{sum(l)}")
@pytest.mark.parametrize("D,W,pad,bias,state,silu", [(8, 4, 0, True, True, True), (24, 3, 8, False, True, True), (37, 4, 5, True, False, False),
                                                     (3, 2, 0, True, True, True), (520, 4, 0, True, True, True), (1040, 4, 0, True, True, True)])
def test_conv_gradients(dtype, gtype, lens, D, W, pad, bias, state, silu):
    say(f"conv bwd {dtype} dy {gtype} N={len(lens)} T={sum(lens)} D={D} W={W}")
    c = make(lens, D, W, dtype, 11, bias, state, pad)
    c["dy"] = c["dy"].to(gtype)
    ref, tol = grads_case(c, lens, silu, dst=state)
    g = kda.conv_bwd(c["x"][None], c["w"], c["bias"], c["dy"][None], c["s0"], c["dst"] if state else None, silu=silu, cu_seqlens=cuts(lens))
    again = kda.conv_bwd(c["x"][None], c["w"], c["bias"], c["dy"][None], c["s0"], c["dst"] if state else None, silu=silu, cu_seqlens=cuts(lens))
    torch.cuda.synchronize()
    check("dx", g["dx"][0], ref[0], tol[0], dtype)
    check("dw", g["dw"], ref[1], tol[1], torch.float32)
    if bias:
        check("dbias", g["dbias"], ref[2], tol[2], torch.float32)
    else:
        assert g["dbias"] is None
    if state:
        check("ds0", g["ds0"], ref[3], tol[3], dtype)
    for k in g:
        assert g[k] is None or torch.equal(g[k], again[k]), k


def test_conv_gradients_batch_equals_packed():
    c = make([70] * 3, 64, 4, torch.bfloat16, 12)
    sh = lambda t: t.reshape(3, 70, 64)
    a = kda.conv_bwd(sh(c["x"]), c["w"], c["bias"], sh(c["dy"]), c["s0"], c["dst"])
    b = kda.conv_bwd(c["x"][None], c["w"], c["bias"], c["dy"][None], c["s0"], c["dst"], cu_seqlens=[0, 70, 140, 210])
    for k in a:
        assert torch.equal(a[k].flatten(), b[k].flatten()), k


def test_conv_captured_and_replayed():
    c = make([40, 33, 90], 64, 4, torch.bfloat16, 13)
    cu = cuts([40, 33, 90])
    x, dy = c["x"][None].contiguous(), c["dy"][None]
    out = {"dx": torch.empty_like(x), "dw": torch.empty_like(c["w"]), "dbias": torch.empty_like(c["bias"]), "ds0": torch.empty_like(c["s0"])}
    y, st, state = torch.empty_like(x), torch.empty_like(c["s0"]), c["s0"].clone()
    ws = torch.empty(kda.lib().kda_conv_bwd_workspace_bytes(1, 163, 64, 4, 3), dtype=torch.uint8, device="cuda")

    def work():
        kda.conv_fwd(x, c["w"], c["bias"], c["s0"], cu_seqlens=cu, st=st, out=y)
        kda.conv_bwd(x, c["w"], c["bias"], dy, c["s0"], c["dst"], cu_seqlens=cu, workspace=ws, out=out)
        kda.conv_step(x[0, :3], c["w"], c["bias"], st, state_out=state)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        work()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        work()
    for k in range(3):
        x.normal_()
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, st, state, out["dx"], out["dw"], out["dbias"], out["ds0"])]
        work()
        torch.cuda.synchronize()
        for a, b in zip(got, (y, st, state, out["dx"], out["dw"], out["dbias"], out["ds0"])):
            assert torch.equal(a, b)


def test_conv_binding_refusals():
    x, w = torch.zeros(2, 8, 16, device="cuda"), torch.zeros(16, 4, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        kda.conv_fwd(x.transpose(1, 2).contiguous().transpose(1, 2), w)
    with pytest.raises(ValueError, match="overlap"):
        kda.conv_fwd(x[:, :1].expand(2, 8, 16)[:1], w)
    with pytest.raises(TypeError):
        kda.conv_fwd(x, w.bfloat16())
    with pytest.raises(ValueError):
        kda.conv_fwd(x, w, s0=torch.zeros(1, 3, 16, device="cuda"))
    with pytest.raises(kda.KDAError):
        kda.conv_fwd(x, torch.zeros(16, 5, device="cuda"))
    with pytest.raises(kda.KDAError):
        kda.conv_fwd(x, w, out=x)
    with pytest.raises(ValueError, match="workspace"):
        kda.conv_bwd(x, w, None, x, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("dtype,D,off", [(torch.float32, 13, 1), (torch.float32, 13, 13)] +
                         [(torch.bfloat16, D, off) for D, off in ((13, 1), (13, 13), (12, 1), (12, 2), (12, 4), (36, 12))])
def test_rows_of_ragged_width_from_any_element(dtype, D, off):
    # states, outputs and gradients as slices of pools that start between two
    # 16-byte places, where a row of D channels is no multiple of 16 bytes
    say(f"conv unaligned {dtype} D={D} off={off}")
    lens, W = [70, 0, 3], 4
    c = make(lens, D, W, dtype, 14)
    cu, x = cuts(lens), c["x"][None]
    gtypes = [dtype] if dtype == torch.float32 else [dtype, torch.float32]

    def shifted(t):
        pool = torch.full((t.numel() + off + 8,), 7, dtype=t.dtype, device="cuda")
        s = pool[off:off + t.numel()].view(t.shape)
        s.copy_(t)
        return s
    y, st = kda.conv_fwd(x, c["w"], c["bias"], c["s0"], cu_seqlens=cu)
    y2, st2 = kda.conv_fwd(shifted(x), c["w"], c["bias"], shifted(c["s0"]), cu_seqlens=cu, st=shifted(st), out=shifted(y))
    assert torch.equal(y, y2) and torch.equal(st, st2)
    one = x[0, :3].contiguous()
    y1, s1 = kda.conv_step(one, c["w"], c["bias"], st.clone()), shifted(st)
    assert torch.equal(kda.conv_step(shifted(one), c["w"], c["bias"], s1, out=shifted(y1)), y1)
    for gt in gtypes:
        if D * gt.itemsize % 16 == 0:
            continue
        dy = c["dy"][None].to(gt)
        g = kda.conv_bwd(x, c["w"], c["bias"], dy, c["s0"], c["dst"], cu_seqlens=cu)
        out = {n: shifted(t) if n in ("dx", "ds0") else torch.empty_like(t) for n, t in g.items()}
        kda.conv_bwd(shifted(x), c["w"], c["bias"], shifted(dy), shifted(c["s0"]), shifted(c["dst"]), cu_seqlens=cu, out=out)
        for n in g:   # (four channels a thread and one add in another order)
            if n in ("dx", "ds0"):
                assert torch.equal(g[n], out[n]), n
        ref, tol = grads_case(dict(c, dy=dy[0]), lens, True, True)
        check("dw", out["dw"], ref[1], tol[1], torch.float32)
        check("dbias", out["dbias"], ref[2], tol[2], torch.float32)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [64, 37])
def test_in_place_states_of_more_sequences_than_a_launch_holds(dtype, D):
    lens = [3] * 126 + [60, 0, 300] + [2, 0] * 60 + [70] + [1] * 10
    c = make(lens, D, 4, dtype, 15)
    want = kda.conv_fwd(c["x"][None], c["w"], c["bias"], c["s0"], cu_seqlens=cuts(lens))
    state = c["s0"].clone()
    y, _ = kda.conv_fwd(c["x"][None], c["w"], c["bias"], state, st=state, cu_seqlens=cuts(lens))
    assert torch.equal(y, want[0]) and torch.equal(state, want[1])
