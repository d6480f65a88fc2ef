"""GPU parity of the gated linear recurrence (kda_lru_fwd, kda_lru_step,
kda_lru_bwd) against the fp64 oracle (oracle/block.py).

Tolerances, u = 2^-24.  A decay a is off by 4 u and by 8 u |g| through its
exponent (gate: exponential, reciprocal and two products), an input u_t by 40 u
|u_t| (two gates, the root of 1 - a^2, whose first term is off by 50 u where the
series ends).  A state in any order of joining runs: two roundings a token.  So
the error of h_t is at most E_t = a E_{t-1} + (4 + 8 |g|) u a H_{t-1} + 40 u |u_t|
+ 2 u H_t with H_t = a H_{t-1} + |u_t|, and likewise F_t for l_t = dL/dh_t with
L_t = |dy_t| + a L_{t+1}.  Products of them add, 100 u for their gates; each
output then rounds by h = finfo.eps / 2.  dc sums at most 16 tokens of a run and
8 runs in fp32 (24 u), parts in 64 bits.  1 - Sigmoid is a difference: the
Sigmoid is off by 2 u of itself at most and the difference rounds by u / 2, 3 u
together, of 1 and not of the difference.
"""
import numpy as np
import pytest
import torch

from gated_delta_rule_96_amd import kda
from kda_testutil import cast, say
from oracle import block

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
DTYPES = [F32, BF]


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def dev(a, dtype=F32):
    return None if a is None else cast(a, dtype).cuda()


def check(name, got, want, tol, dtype):
    h = torch.finfo(dtype).eps / 2
    lim = tol * (1 + h) + h * np.abs(want) + 2.0 ** -133
    bad = ~(np.abs(f64(got) - want) <= lim)
    assert not bad.any(), (name, int(bad.sum()), float(np.max(np.abs(f64(got) - want) / lim)))


def cuts(lens):
    return [0] + [int(v) for v in np.cumsum(lens)]


def make(lens, D, dtype, seed, gate=True, igate=True, state=True, pad=0, slow=False):
    """Packed rows [1, sum of lens, D] as slices of one wider tensor (pad), or tensors of their own."""
    r = np.random.default_rng(seed)
    T, N = sum(lens), len(lens)
    lo, hi = (0.9, 0.999) if slow else (0.3, 0.999)
    x = r.standard_normal((1, T, D))
    rec = r.standard_normal((1, T, D)) if gate else np.log(r.uniform(lo, hi, (1, T, D)))
    inp = r.standard_normal((1, T, D)) if igate else None
    parts = [x, rec] + ([inp] if igate else [])
    if pad:
        row = dev(np.concatenate(parts + [np.full((1, T, pad), np.nan)], -1), dtype)
        parts = [row[..., k * D:(k + 1) * D] for k in range(len(parts))]
    else:
        parts = [dev(p, dtype) for p in parts]
    c = dev(-np.log(r.uniform(lo, hi, D))) if gate else None
    return dict(x=parts[0], r=parts[1], i=parts[2] if igate else None, c=c, h0=dev(r.standard_normal((N, D))) if state else None,
                dy=dev(r.standard_normal((1, T, D)), dtype), dht=dev(r.standard_normal((N, D))) if state else None)


def oracle(k, lens, unit, back=False):
    """Results and tolerances of every sequence, joined."""
    x, r, i, c, h0, dy, dht = (f64(k[n]) for n in ("x", "r", "i", "c", "h0", "dy", "dht"))
    cu, D = cuts(lens), x.shape[-1]
    out = {n: [] for n in ("y", "ty", "ht", "tht", "dx", "tdx", "dr", "tdr", "di", "tdi", "dh0", "tdh0")}
    dc, tdc = np.zeros(D), np.zeros(D)
    for n, (lo, hi) in enumerate(zip(cu, cu[1:])):
        s = [v[0, lo:hi] if v is not None else None for v in (x, r, i)]
        start = np.zeros(D) if h0 is None else h0[n]
        y, ht = block.lru_fwd(*s, c, start, unit)
        g, a, m, si = block.lru_gates(*s, c, unit)
        u = np.abs(m * si * s[0])
        H, E = np.abs(start), np.zeros(D)
        ea = (4 + 8 * np.abs(np.where(a > 0, g, 0.0))) * U
        Hb, Eb, Ey = np.empty_like(y), np.empty_like(y), np.empty_like(y)
        for t in range(hi - lo):
            Hb[t], Eb[t] = H, E
            E = a[t] * E + ea[t] * a[t] * H + 40 * U * u[t]
            H = a[t] * H + u[t]
            E = E + 2 * U * H
            Ey[t] = E
        for name, v in (("y", y), ("ty", Ey), ("ht", ht), ("tht", E)):
            out[name].append(v)
        if not back:
            continue
        d = dy[0, lo:hi]
        dx, dr, di, dcn, dh0, lam = block.lru_bwd(*s, c, start, d, None if dht is None else dht[n], unit)
        L, e, F = np.empty_like(lam), np.abs(dht[n]) if dht is not None else np.zeros(D), np.zeros(D)
        Fl = np.empty_like(lam)
        for t in range(hi - lo - 1, -1, -1):
            L[t] = np.abs(d[t]) + e
            Fl[t] = F + 2 * U * L[t]
            F = a[t] * Fl[t] + ea[t] * a[t] * L[t]
            e = a[t] * L[t]
        ms = m * si
        tx = Fl * ms + 100 * U * L * ms
        with np.errstate(divide="ignore", invalid="ignore"):
            back2 = np.where(m > 0, si * np.abs(s[0]) * a * a / m, 0.0) if unit else np.zeros_like(a)
        before = np.concatenate([start[None], y])[:-1]
        tg = a * (Fl * np.abs(before) + L * Eb + 100 * U * L * Hb) + back2 * (Fl + 100 * U * L)
        sg = np.abs(g) * block.sigmoid(-s[1]) if c is not None else np.ones_like(g)
        size = L * (a * Hb + back2)
        for name, v in (("dx", dx), ("tdx", tx), ("dr", dr), ("tdr", (tg + 20 * U * size) * sg + (3 * U * size * np.abs(g) if c is not None else 0.0)), ("dh0", dh0), ("tdh0", F)):
            out[name].append(v)
        if i is not None:
            out["di"].append(di)
            out["tdi"].append(((tx + 20 * U * L * ms) * block.sigmoid(-s[2]) + 3 * U * L * ms) * np.abs(s[0]))
        if c is not None:
            sr = block.sigmoid(s[1])
            dc += dcn
            tdc += ((tg + 30 * U * size) * sr).sum(0)
    res = {n: (np.stack(v) if n in ("ht", "tht", "dh0", "tdh0") else np.concatenate(v)) if v else None for n, v in out.items()}
    res["dc"], res["tdc"] = (dc, tdc) if c is not None else (None, None)
    return res


def compare_grads(k, got, want, dtype):
    for n in ("dx", "dr", "di"):
        if want[n] is None:
            assert got[n] is None
        else:
            check(n, got[n].reshape(want[n].shape), want[n], want["t" + n], dtype)
    if want["dc"] is None:
        assert got["dc"] is None
    else:
        check("dc", got["dc"], want["dc"], want["tdc"], F32)
    if k["h0"] is not None:
        check("dh0", got["dh0"], want["dh0"], want["tdh0"], F32)


LENS = [[1], [2], [15], [16], [17], [64], [127], [128], [129], [300], [1, 0, 130, 3], [0, 0, 5], [256, 128, 1, 0, 511], [700], [40] * 9]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_prompts_and_gradients(dtype, lens):
    for D, gate, igate, unit, state, pad in ((128, True, True, True, True, 0), (130, True, False, True, True, 2), (33, False, True, False, False, 5),
                                             (7, True, True, False, True, 0), (384, False, False, True, True, 8), (1, True, True, True, False, 0)):
        say(f"recurrence {dtype} {lens} D={D} gate={gate} igate={igate} unit={unit} pad={pad}")
        k = make(lens, D, dtype, 31 + D, gate, igate, state, pad)
        args, kw = (k["x"], k["r"], k["i"], k["c"]), dict(unit=unit, cu_seqlens=cuts(lens))
        y, ht = kda.lru_fwd(*args, k["h0"], **kw)
        g = kda.lru_bwd(*args, k["dy"], k["h0"], k["dht"], **kw)
        y2, ht2 = kda.lru_fwd(*args, k["h0"], **kw)
        g2 = kda.lru_bwd(*args, k["dy"], k["h0"], k["dht"], **kw)
        torch.cuda.synchronize()
        want = oracle(k, lens, unit, back=True)
        check("y", y[0], want["y"], want["ty"], dtype)
        check("ht", ht, want["ht"], want["tht"], F32)
        compare_grads(k, g, want, dtype)
        assert torch.equal(y, y2) and torch.equal(ht, ht2)
        assert all(g[n] is None and g2[n] is None or torch.equal(g[n], g2[n]) for n in g)


@pytest.mark.parametrize("dtype", DTYPES)
def test_long_prompts_with_long_memory(dtype):
    lens = [5000, 3001]
    k = make(lens, 192, dtype, 41, slow=True)
    kw = dict(cu_seqlens=cuts(lens))
    y, ht = kda.lru_fwd(k["x"], k["r"], k["i"], k["c"], k["h0"], **kw)
    g = kda.lru_bwd(k["x"], k["r"], k["i"], k["c"], k["dy"], k["h0"], k["dht"], **kw)
    want = oracle(k, lens, True, back=True)
    check("y", y[0], want["y"], want["ty"], dtype)
    check("ht", ht, want["ht"], want["tht"], F32)
    compare_grads(k, g, want, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,T,D", [(3, 200, 130), (2, 1, 64), (70, 5, 34), (1, 1000, 4100)])
def test_batches_equal_their_sequences(dtype, B, T, D):
    k = make([T] * B, D, dtype, 51)
    rows = {n: k[n].reshape(B, T, D) for n in ("x", "r", "i", "dy")}
    y, ht = kda.lru_fwd(rows["x"], rows["r"], rows["i"], k["c"], k["h0"])
    g = kda.lru_bwd(rows["x"], rows["r"], rows["i"], k["c"], rows["dy"], k["h0"], k["dht"])
    want = oracle(k, [T] * B, True, back=True)
    check("y", y.reshape(B * T, D), want["y"], want["ty"], dtype)
    check("ht", ht, want["ht"], want["tht"], F32)
    compare_grads(k, g, want, dtype)


def test_more_sequences_than_one_launch_carries():
    lens = [(7 * n) % 300 for n in range(300)]
    k = make(lens, 40, BF, 61)
    kw = dict(cu_seqlens=cuts(lens))
    y, ht = kda.lru_fwd(k["x"], k["r"], k["i"], k["c"], k["h0"], **kw)
    g = kda.lru_bwd(k["x"], k["r"], k["i"], k["c"], k["dy"], k["h0"], k["dht"], **kw)
    want = oracle(k, lens, True, back=True)
    check("y", y[0], want["y"], want["ty"], BF)
    check("ht", ht, want["ht"], want["tht"], F32)
    compare_grads(k, g, want, BF)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,D,gate,igate,unit,pad", [(1, 1, True, True, True, 0), (5, 130, True, True, True, 2), (256, 64, False, False, False, 0),
                                                     (3, 7, True, False, True, 3), (2, 4096, False, True, True, 0)])
def test_token_step(dtype, B, D, gate, igate, unit, pad):
    lens = [1] * B
    k = make(lens, D, dtype, 71, gate, igate, True, pad)
    x, r, i = (k[n][0] if k[n] is not None else None for n in ("x", "r", "i"))
    want = oracle(k, lens, unit)
    state, kept = k["h0"].clone(), k["h0"].clone()
    so = torch.empty_like(kept)
    y2 = kda.lru_step(x, r, i, k["c"], kept, unit=unit, state_out=so)
    y = kda.lru_step(x, r, i, k["c"], state, unit=unit)
    yp, hp = kda.lru_fwd(x[:, None], r[:, None], None if i is None else i[:, None], k["c"], k["h0"], unit=unit)
    torch.cuda.synchronize()
    check("y", y, want["y"], want["ty"], dtype)
    check("state", state, want["ht"], want["tht"], F32)
    assert torch.equal(y, y2) and torch.equal(state, so) and torch.equal(kept, k["h0"])
    assert torch.equal(y, yp[:, 0]) and torch.equal(state, hp)


@pytest.mark.parametrize("dtype", DTYPES)
def test_carry_in_place_and_tokens_behind_a_prompt(dtype):
    k = make([333], 66, dtype, 81)
    args = lambda lo, hi: (k["x"][:, lo:hi], k["r"][:, lo:hi], k["i"][:, lo:hi], k["c"])
    state, ys = k["h0"].clone(), []
    for lo, hi in ((0, 130), (130, 131), (131, 320)):
        y, st = kda.lru_fwd(*args(lo, hi), state, ht=state)
        assert st is state
        ys.append(y)
    for t in range(320, 333):
        ys.append(kda.lru_step(k["x"][:, t], k["r"][:, t], k["i"][:, t], k["c"], state)[:, None])
    torch.cuda.synchronize()
    want = oracle(k, [333], True)
    check("y", torch.cat(ys, 1)[0], want["y"], want["ty"], dtype)
    check("state", state, want["ht"], want["tht"], F32)


def test_resets_open_gates_and_values_that_are_not_finite():
    T, D = 400, 6
    k = make([T], D, F32, 91, gate=False, igate=False)
    g = k["r"].clone()
    g[0, 150, 0] = float("-inf")      # starts anew
    g[0, 37, 1] = 0.0                 # keeps the state, m = 0
    x = k["x"].clone()
    x[0, 200, 2] = float("nan")
    x[0, 250, 3] = float("inf")
    g[0, 300, 4] = float("nan")
    for unit in (False, True):
        k2 = dict(k, x=x, r=g)
        y, ht = kda.lru_fwd(x, g, None, None, k["h0"], unit=unit)
        gr = kda.lru_bwd(x, g, None, None, k["dy"], k["h0"], k["dht"], unit=unit)
        torch.cuda.synchronize()
        clean = dict(k, x=k["x"], r=torch.where(torch.isnan(g), k["r"], g))
        want = oracle(clean, [T], unit, back=True)
        live = np.ones((T, D), bool)
        live[200:, 2], live[250:, 3], live[300:, 4] = False, False, False
        ok = lambda a, m: np.where(m, a, 0.0)
        got = f64(y[0])
        assert not np.isfinite(got[~live]).any()
        check("y", torch.from_numpy(ok(got, live)), ok(want["y"], live), ok(want["ty"], live), F32)
        for c in (0, 1, 5):
            for n in ("dx", "dr"):
                check(n, gr[n][0, :, c], want[n][:, c], want["t" + n][:, c], F32)
        # a bad input token gives bad gradients of its own and later tokens at most (its decay is sound)
        assert torch.isfinite(gr["dx"][0, :, 2:4]).sum() >= 2 * 199
        assert np.isfinite(f64(gr["dh0"])[0, [0, 1, 2, 3, 5]]).all() and torch.isnan(gr["dh0"][0, 4])


def test_gradient_of_the_forward_against_differences():
    # central differences of the fp32 forward: step e off by e^2 of the third
    # derivative (below 8 S for these gates), values by 100 u S, S = sum |dy| H
    k = make([40], 16, F32, 101)
    r = np.random.default_rng(102)
    want = oracle(k, [40], True, back=True)
    S = float(sum(np.abs(f64(k["dy"]))[0].sum(0) * 10)) + 1
    e = 2.0 ** -6
    g = kda.lru_bwd(k["x"], k["r"], k["i"], k["c"], k["dy"], k["h0"], None)
    for n, gn in (("x", "dx"), ("r", "dr"), ("i", "di"), ("c", "dc"), ("h0", "dh0")):
        d = dev(r.standard_normal(tuple(k[n].shape)))
        if n == "c":
            d = d * k["c"]

        def f(s):
            v = dict(k, **{n: k[n] + s * d})
            y, _ = kda.lru_fwd(v["x"], v["r"], v["i"], v["c"], v["h0"])
            return float((y.double() * k["dy"].double()).sum())
        slope = (f(e) - f(-e)) / (2 * e)
        got = float((g[gn].double() * d.double()).sum())
        assert abs(slope - got) <= 8 * e * e * S + 200 * U * S / e, n
    assert want["dc"] is not None


def test_odd_starts_and_neighbours_stay():
    # rows that start on an odd element, outputs with guards around them
    T, D = 150, 33
    k = make([T], D, BF, 111, pad=0)
    odd = lambda t: torch.cat([torch.zeros(1, dtype=t.dtype, device="cuda"), t.reshape(-1)])[1:].view(t.shape)
    buf = torch.full((T * D + 64,), 5.0, dtype=BF, device="cuda")
    y, ht = kda.lru_fwd(odd(k["x"]), odd(k["r"]), odd(k["i"]), k["c"], k["h0"], out=buf[1:1 + T * D].view(1, T, D))
    want, _ = kda.lru_fwd(k["x"], k["r"], k["i"], k["c"], k["h0"])
    assert torch.equal(y, want) and bool((buf[:1] == 5).all()) and bool((buf[1 + T * D:] == 5).all())


def test_refusals():
    x = torch.zeros(1, 4, 8, device="cuda")
    c = torch.zeros(8, device="cuda")
    with pytest.raises(ValueError, match="c must be"):
        kda.lru_fwd(x, x, None, c[:4])
    with pytest.raises(ValueError, match="rise"):
        kda.lru_fwd(x, x, cu_seqlens=[0, 3])
    with pytest.raises(kda.KDAError) as e:
        kda.lru_fwd(x, x, out=x)
    assert e.value.status == kda.KDA_ERR_OVERLAP
    with pytest.raises(ValueError, match="workspace"):
        kda.lru_fwd(x, x, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError, match="h0"):
        kda.lru_fwd(x, x, None, None, torch.zeros(1, 8, device="cuda", dtype=torch.float64))
    with pytest.raises(kda.KDAError):
        kda.lru_bwd(x, x, None, None, x, out=dict(dx=torch.empty_like(x), dr=torch.empty_like(x), di=None, dc=torch.empty(8, device="cuda"), dh0=None))


@pytest.mark.parametrize("dtype", DTYPES)
def test_sequences_of_many_parts(dtype):
    # hundreds of parts of few channels: the state comes from far back, and the
    # gradients' chain takes more runs of them
    lens = [20000, 9, 300]
    say(f"recurrence {dtype} {lens} D=48")
    k = make(lens, 48, dtype, 121, slow=True)
    kw = dict(cu_seqlens=cuts(lens))
    y, ht = kda.lru_fwd(k["x"], k["r"], k["i"], k["c"], k["h0"], **kw)
    g = kda.lru_bwd(k["x"], k["r"], k["i"], k["c"], k["dy"], k["h0"], k["dht"], **kw)
    torch.cuda.synchronize()
    want = oracle(k, lens, True, back=True)
    check("y", y[0], want["y"], want["ty"], dtype)
    check("ht", ht, want["ht"], want["tht"], F32)
    compare_grads(k, g, want, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
def test_bits_do_not_depend_on_how_the_state_was_found(dtype):
    # channels are on their own: many of them (each part looks back over a few
    # parts) and a few of them (over many) give the same bits, every time
    B, T, D = 2, 12000, 1300
    say(f"recurrence {dtype} {B} x {T} x {D}")
    x, r, i = (dev(np.random.default_rng(s).standard_normal((B, T, D)), dtype) for s in (131, 132, 133))
    c, h0 = dev(-np.log(np.random.default_rng(134).uniform(0.9, 0.999, D))), dev(np.random.default_rng(135).standard_normal((B, D)))
    y, ht = kda.lru_fwd(x, r, i, c, h0)
    for n in range(4):
        lo = 256 * n
        few = [t[..., lo:lo + 256] for t in (x, r, i)]
        yf, hf = kda.lru_fwd(*few, c[lo:lo + 256].clone(), h0[:, lo:lo + 256].contiguous())
        y2, ht2 = kda.lru_fwd(x, r, i, c, h0)
        torch.cuda.synchronize()
        assert torch.equal(yf, y[..., lo:lo + 256]) and torch.equal(hf, ht[:, lo:lo + 256])
        assert torch.equal(y2, y) and torch.equal(ht2, ht)
