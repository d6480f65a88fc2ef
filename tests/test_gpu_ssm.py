"""GPU parity of the state space scan (kda_ssm_fwd_chunked, kda_ssm_step)
against the fp64 oracle (oracle/mix.py) on the cast inputs.

Tolerances, per element, u = 2^-24, h = finfo.eps / 2 of the type.  `size` is
the scan on absolute values: every product that reaches an output is one of
its terms.  fp32 arithmetic: a chunk adds at most 64 (tokens) + 128 (state
channels) terms, a state passes one product and one addition per chunk, a
decay factor exp2 of an exponent e rounded to 32 bits is off by (|e| u + 2 u)
with 2^e |e| <= 0.54 of the term it weighs, a step size by 8 u: at most (250 +
4 chunks) u size.  bf16 adds: the operands M and S of y rounded once (h each)
and the 32-bit decay sums in M, off by 2 u max|cum|; the state's update keeps
24 bits.  The output's own rounding: h |y|.
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


def make(lens, H, G, dk, dv, dtype, seed, skip=True, soft=True, state=True, packed_rows=False, rate=16.0, slow=False):
    r = np.random.default_rng(seed)
    T, N = sum(lens), len(lens)
    widths = [H * dv, G * dk, G * dk, H]
    wide = r.standard_normal((T, sum(widths)))
    parts = np.split(wide, np.cumsum(widths)[:-1], 1)
    step = np.exp(r.uniform(np.log(1e-3), np.log(0.1), H)) * (0.01 if slow else 1.0)
    bias = step + np.log(-np.expm1(-step))
    raw = 0.5 * parts[3] + (0 if soft else bias)
    if not soft:
        raw = mix.softplus(raw)
    t = [cast(p, dtype).cuda() for p in (parts[0], parts[1], parts[2], raw)]
    if packed_rows:   # slices of one tensor: x, B, C and then the step sizes
        one = torch.cat(t, 1)
        one = torch.nn.functional.pad(one, (0, (-one.shape[1]) % 8))
        t = [one[:, a:a + w] for a, w in zip(np.cumsum([0] + widths[:-1]).tolist(), widths)]
    v = lambda a: cast(a, torch.float32).cuda()
    return dict(x=t[0].unflatten(1, (H, dv)), B=t[1].unflatten(1, (G, dk)), C=t[2].unflatten(1, (G, dk)), dt=t[3],
                A=v(-r.uniform(1, rate, H)), bias=v(bias) if soft else None, D=v(r.standard_normal(H)) if skip else None,
                h0=v(0.5 * r.standard_normal((N, H, dk, dv))) if state else None, soft=soft)


def cuts(lens):
    return np.concatenate([[0], np.cumsum(lens)]).tolist()


def oracle(c, lens, dtype):
    cu, ys, hs, ty, th = cuts(lens), [], [], [], []
    dt = f64(c["dt"]) + (0 if c["bias"] is None else f64(c["bias"]))
    dt = mix.softplus(dt) if c["soft"] else dt
    for i, n in enumerate(lens):
        sl = slice(cu[i], cu[i + 1])
        y, h, size, zt = mix.ssm_seq(f64(c["x"])[sl], f64(c["dt"])[sl], f64(c["A"]), f64(c["B"])[sl], f64(c["C"])[sl],
                                     None if c["h0"] is None else f64(c["h0"])[i], f64(c["D"]), f64(c["bias"]), c["soft"])
        k = (250 + 4 * (n // 64 + 1)) * U
        m = max((np.abs((dt[sl] * f64(c["A"]))[a:a + 64]).sum(0).max() for a in range(0, n, 64)), default=0.0) * 1.45
        ys.append(y)
        hs.append(h)
        ty.append(size * (k + (2 ** -8 * 1.01 + 2 * m * U if dtype == torch.bfloat16 else 0)))
        th.append(zt * k)
    return np.concatenate(ys), np.stack(hs), np.concatenate(ty), np.stack(th)


def check(name, got, want, tol, dtype):
    h = torch.finfo(dtype).eps / 2
    lim = tol * (1 + h) + h * np.abs(want) + 1e-37
    bad = ~(np.abs(f64(got) - want) <= lim)
    assert not bad.any(), (name, int(bad.sum()), float(np.nanmax(np.abs(f64(got) - want) / lim)), np.argwhere(bad)[:3].tolist())


def call(c, lens=None, B=None, **kw):
    sh = (lambda t: t[None]) if B is None else (lambda t: t.unflatten(0, (B, -1)))
    return kda.ssm_fwd_chunked(sh(c["x"]), sh(c["dt"]), c["A"], sh(c["B"]), sh(c["C"]), c["h0"], D=c["D"], dt_bias=c["bias"], softplus=c["soft"],
                               cu_seqlens=None if B else cuts(lens), **kw)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens", [[1], [63], [64], [65], [5, 0, 1, 130, 64, 0], [300, 700], [0, 2], [2] * 131, [3] * 130 + [800, 2]], ids=lambda l: f"{len(l)}x{sum(l)}")
@pytest.mark.parametrize("H,G,dk,dv,skip,soft,state,rows", [(2, 1, 64, 64, True, True, True, False), (4, 2, 128, 128, False, False, True, False),
                                                            (3, 3, 128, 64, True, True, False, True), (2, 2, 64, 128, True, True, True, True)])
def test_packed(dtype, lens, H, G, dk, dv, skip, soft, state, rows):
    say(f"ssm packed {dtype} N={len(lens)} T={sum(lens)} H={H} G={G} dk={dk} dv={dv}")
    c = make(lens, H, G, dk, dv, dtype, 31, skip, soft, state, rows)
    y_ref, h_ref, ty, th = oracle(c, lens, dtype)
    y, ht = call(c, lens)
    torch.cuda.synchronize()
    check("y", y[0], y_ref, ty, dtype)
    check("ht", ht, h_ref, th, torch.float32)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,T,H,G,slow", [(1, 2500, 4, 1, False), (3, 600, 2, 2, True), (2, 257, 1, 1, True), (2, 1100, 2, 2, True)])
def test_parts_of_long_sequences_and_in_place_state(dtype, B, T, H, G, slow):
    # parts of 256 tokens: chained states, h0 replaced in place by ht
    say(f"ssm batch {dtype} B={B} T={T} H={H} G={G}")
    c = make([T] * B, H, G, 128, 128, dtype, 32, rate=2.0, slow=slow)
    y_ref, h_ref, ty, th = oracle(c, [T] * B, dtype)
    c["h0"] = c["h0"].clone()
    first = call(c, B=B)
    y, ht = call(c, B=B, ht=c["h0"])
    torch.cuda.synchronize()
    assert ht.data_ptr() == c["h0"].data_ptr() and torch.equal(first[0], y) and torch.equal(first[1], ht)
    check("y", y.flatten(0, 1), y_ref, ty, dtype)
    check("ht", ht, h_ref, th, torch.float32)


@pytest.mark.parametrize("dtype", DTYPES)
def test_many_heads_and_strong_decay(dtype):
    # decays that leave nothing of the state within a chunk, and step sizes of zero
    c = make([200], 40, 4, 64, 64, dtype, 33, rate=400.0)
    c["dt"][:7] = -100.0 if c["soft"] else 0.0
    y_ref, h_ref, ty, th = oracle(c, [200], dtype)
    y, ht = call(c, [200])
    torch.cuda.synchronize()
    check("y", y[0], y_ref, ty, dtype)
    check("ht", ht, h_ref, th, torch.float32)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,H,G,dk,dv,skip,soft", [(1, 1, 1, 64, 64, True, True), (3, 4, 2, 128, 64, False, True), (5, 3, 1, 64, 128, True, False),
                                                   (2, 32, 1, 128, 128, True, True)])
def test_step_continues_the_prompt(dtype, B, H, G, dk, dv, skip, soft):
    say(f"ssm step {dtype} B={B} H={H} G={G} dk={dk} dv={dv}")
    T = 70
    c = make([T] * B, H, G, dk, dv, dtype, 34, skip, soft, True, True)
    y_ref, h_ref, ty, th = oracle(c, [T] * B, dtype)
    sh = lambda t, a, b: t.unflatten(0, (B, T))[:, a:b]
    part = lambda a, b: dict(c, **{n: sh(c[n], a, b).flatten(0, 1) for n in ("x", "dt", "B", "C")})
    y, state = call(part(0, 66), B=B)
    ys = [y]
    for t in range(66, T):
        a = [sh(c[n], t, t + 1)[:, 0] for n in ("x", "dt", "B", "C")]
        kw = dict(D=c["D"], dt_bias=c["bias"], softplus=c["soft"])
        kept, nxt = state.clone(), torch.full_like(state, float("nan"))
        y1 = kda.ssm_step(a[0], a[1], c["A"], a[2], a[3], state, state_out=nxt, **kw)
        assert torch.equal(kept, state)
        y2 = kda.ssm_step(a[0], a[1], c["A"], a[2], a[3], state, **kw)
        assert torch.equal(y1, y2) and torch.equal(nxt, state)
        ys.append(y1[:, None])
    torch.cuda.synchronize()
    check("y", torch.cat(ys, 1).flatten(0, 1), y_ref, ty, dtype)
    check("state", state, h_ref, th, torch.float32)


def test_rows_behind_and_other_sequences_untouched():
    # a NaN token changes its own sequence alone; rows of y behind T stay
    lens = [40, 90, 30]
    c = make(lens, 2, 1, 64, 64, torch.bfloat16, 35)
    y0, h0 = call(c, lens)
    c["x"][50] = float("nan")
    big = torch.full((1, 200, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    y, ht = call(c, lens, out=big[:, :160])
    assert torch.equal(y[0, :50], y0[0, :50]) and torch.equal(y[0, 130:], y0[0, 130:]) and torch.isnan(y[0, 51:130]).all()
    assert torch.equal(ht[0], h0[0]) and torch.equal(ht[2], h0[2]) and (big[0, 160:] == 7).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("name", ["x", "B", "C", "dt"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf"), "lowest"])
def test_a_bad_token_stays_out_of_the_tokens_before_it(dtype, name, bad):
    # token 170 is in the middle of the second chunk of 64 of its sequence: the
    # tokens before it and the other sequences do not see it
    say(f"ssm bad token {dtype} {name} {bad}")
    lens = [100, 600, 30]
    c = make(lens, 2, 1, 64, 64, dtype, 38, rate=2.0)
    y_ref, _, ty, _ = oracle(c, lens, dtype)
    y0, h0 = call(c, lens)
    c[name][170] = torch.finfo(dtype).min if bad == "lowest" else bad
    y, ht = call(c, lens)
    assert torch.equal(y[0, :164], y0[0, :164]) and torch.equal(y[0, 700:], y0[0, 700:])
    check("y before", y[0, 164:170], y_ref[164:170], ty[164:170], dtype)   # (a chunk with a bad x sums in another order)
    assert torch.equal(ht[0], h0[0]) and torch.equal(ht[2], h0[2])
    if name == "dt" and bad in ("lowest", float("-inf")):   # Softplus of it is zero: the token leaves the state alone
        assert torch.isfinite(y).all() and torch.isfinite(ht).all()
        y_ref, h_ref, ty, th = oracle(dict(c, dt=c["dt"].clamp(min=-1e3)), lens, dtype)
        check("y", y[0], y_ref, ty, dtype)
        check("ht", ht, h_ref, th, torch.float32)
    elif name == "C" and bad != "lowest":
        assert not torch.isfinite(y[0, 170]).any() and torch.equal(y[0, 171:], y0[0, 171:]) and torch.equal(ht, h0)
    elif bad != "lowest":
        assert not torch.isfinite(y[0, 170]).all() and not torch.isfinite(ht[1]).all()


def test_captured_and_replayed():
    lens = [700, 1, 0, 260]
    c = make(lens, 2, 1, 128, 128, torch.bfloat16, 36)
    ws = torch.empty(kda.lib().kda_ssm_workspace_bytes(1, 961, 2, 128, 128, 1), dtype=torch.uint8, device="cuda")
    y, ht, nxt = torch.empty((1, 961, 2, 128), dtype=torch.bfloat16, device="cuda"), torch.empty_like(c["h0"]), torch.empty_like(c["h0"])

    def work():
        call(c, lens, ht=ht, out=y, workspace=ws)
        kda.ssm_step(c["x"][:4], c["dt"][:4], c["A"], c["B"][:4], c["C"][:4], ht, D=c["D"], dt_bias=c["bias"], softplus=True, state_out=nxt)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        work()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        work()
    for _ in range(3):
        c["x"].normal_()
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, ht, nxt)]
        work()
        torch.cuda.synchronize()
        for a, b in zip(got, (y, ht, nxt)):
            assert torch.equal(a, b)


def test_refusals_of_the_binding():
    c = make([8], 2, 1, 64, 64, torch.float32, 37)
    with pytest.raises(ValueError):
        kda.ssm_fwd_chunked(c["x"][None], c["dt"][None], c["A"][:1], c["B"][None], c["C"][None])
    with pytest.raises(TypeError):
        kda.ssm_fwd_chunked(c["x"][None], c["dt"][None].bfloat16(), c["A"], c["B"][None], c["C"][None])
    with pytest.raises(ValueError):
        kda.ssm_fwd_chunked(c["x"][None], c["dt"][None], c["A"], c["B"][None], c["C"][None, :7])
    with pytest.raises(kda.KDAError):
        kda.ssm_fwd_chunked(c["x"][None, ..., :32].contiguous(), c["dt"][None], c["A"], c["B"][None], c["C"][None])


def reset_case(dtype, big, soft, seed):
    """Small steps with two resetting tokens (a huge step, x = 0) in mid-chunk."""
    c = make([200], 2, 1, 64, 128, dtype, seed, soft=False, rate=2.0)
    c["A"].fill_(-16.0)
    c["dt"].copy_(0.005 * torch.rand(c["dt"].shape, device="cuda") + 0.002)
    if soft:   # the raw values whose Softplus the steps are
        c["dt"].copy_(torch.log(torch.expm1(c["dt"].float())))
        c["soft"] = True
    for t in (80, 150):
        c["dt"][t] = big
        c["x"][t] = 0
        if big > 1e30:   # (their product with B would be out of range)
            c["B"][t] = 0
    return c


def reset_check(c, dtype):
    # As at the head of the file, without the term for 32-bit decay sums: a
    # step's exponent |e| costs its own rounding alone, 0.54 u at most.
    y_ref, h_ref, size, zt = mix.ssm_seq(f64(c["x"]), f64(c["dt"]), f64(c["A"]), f64(c["B"]), f64(c["C"]), f64(c["h0"])[0], f64(c["D"]), None, c["soft"])
    k = (250 + 4 * 4) * U
    ty, th = size * (k + (2 ** -8 * 1.01 if dtype == torch.bfloat16 else 0)), zt * k
    y, ht = call(c, [200])
    state, ys = c["h0"].clone(), []
    for t in range(200):
        ys.append(kda.ssm_step(c["x"][t:t + 1], c["dt"][t:t + 1], c["A"], c["B"][t:t + 1], c["C"][t:t + 1], state, D=c["D"], softplus=c["soft"]))
    torch.cuda.synchronize()
    check("step", torch.cat(ys), y_ref, ty, dtype)
    check("state", state[0], h_ref, th, torch.float32)
    check("ht", ht[0], h_ref, th, torch.float32)
    check("y", y[0], y_ref, ty, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("soft", [False, True])
@pytest.mark.parametrize("big", [2.0 ** 13, 2.0 ** 17, 2.0 ** 20])
def test_small_steps_behind_a_reset(dtype, soft, big):
    # exp(dt A) of a huge step leaves nothing of the state; the tokens behind it
    # in the chunk keep their own small decays
    say(f"ssm reset {dtype} dt={big} soft={soft}")
    reset_check(reset_case(dtype, big, soft, 39), dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("soft", [False, True])
def test_small_steps_behind_a_reset_of_the_largest_step(dtype, soft):
    say(f"ssm reset {dtype} dt=max soft={soft}")
    reset_check(reset_case(dtype, torch.finfo(dtype).max, soft, 40), dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("big", [2.0 ** 17, "max"])
def test_resets_in_a_sequence_of_several_parts(dtype, big):
    # parts of 256 tokens: a reset inside a part, on its first and on its last token
    say(f"ssm reset parts {dtype} dt={big}")
    T = 1300
    c = make([T], 2, 1, 64, 64, dtype, 50, soft=False, rate=2.0)
    c["A"].fill_(-16.0)
    c["dt"].copy_(0.005 * torch.rand(c["dt"].shape, device="cuda") + 0.002)
    for t in (100, 256, 767, 1090):
        c["dt"][t] = torch.finfo(dtype).max if big == "max" else big
        c["x"][t] = 0
        c["B"][t] = 0
    y_ref, h_ref, size, zt = mix.ssm_seq(f64(c["x"]), f64(c["dt"]), f64(c["A"]), f64(c["B"]), f64(c["C"]), f64(c["h0"])[0], f64(c["D"]), None, False)
    k = (250 + 4 * (T // 64 + 1)) * U
    y, ht = call(c, [T])
    torch.cuda.synchronize()
    check("ht", ht[0], h_ref, zt * k, torch.float32)
    check("y", y[0], y_ref, size * (k + (2 ** -8 * 1.01 if dtype == torch.bfloat16 else 0)), dtype)


@pytest.mark.parametrize("dtype", DTYPES)
def test_in_place_states_of_more_sequences_than_a_launch_holds(dtype):
    # 260 sequences, three launches, some cut into parts
    lens = [3] * 126 + [600, 0, 300] + [2, 0] * 60 + [700] + [1] * 10
    say(f"ssm in place {dtype} N={len(lens)}")
    c = make(lens, 2, 1, 64, 64, dtype, 51, rate=2.0)
    want = call(c, lens)
    state = c["h0"].clone()
    y, ht = call(dict(c, h0=state), lens, ht=state)
    assert ht.data_ptr() == state.data_ptr() and torch.equal(y, want[0]) and torch.equal(state, want[1])
