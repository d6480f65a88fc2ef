"""GPU parity of the scan's gradients (kda_ssm_bwd_chunked) against the fp64
oracle (oracle/mix.py, itself held to finite differences) on the cast inputs.

Tolerances, per element, u = 2^-24, h = finfo.eps / 2.  The oracle's "|" sums
hold the size of every product that reaches a gradient.  fp32 arithmetic as
for the forward (tests/test_gpu_ssm.py) along and against the tokens and once
more in the chunk: 3 (250 + 4 chunks) u of that size; sums over tokens (dA, dD,
ddt_bias) are 64-bit sums of fp32 terms.  ddt and dA take differences of a
chunk's sums of the same terms, at most two chunk sums deep: 4 times as much,
of the size of the largest token sum of the sequence for ddt (a chunk's sums
enter every token of it).  bf16 adds one rounding of an operand of dx, dB and
dC: h of the size; ddt, dA, dD, ddt_bias and dh0 take none.
"""
import numpy as np
import pytest
import torch

from gated_delta_rule_96_amd import kda
from kda_testutil import cast, say
from oracle import mix
from test_gpu_ssm import U, DTYPES, check, cuts, f64, make

pytestmark = pytest.mark.gpu
NAMES = ["dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "dh0"]


def oracle(c, lens):
    cu, got = cuts(lens), []
    for i in range(len(lens)):
        sl = slice(cu[i], cu[i + 1])
        got.append(mix.ssm_seq_bwd(f64(c["x"])[sl], f64(c["dt"])[sl], f64(c["A"]), f64(c["B"])[sl], f64(c["C"])[sl], f64(c["dy"])[sl],
                                   None if c["h0"] is None else f64(c["h0"])[i], None if c["dht"] is None else f64(c["dht"])[i], f64(c["D"]),
                                   f64(c["bias"]), c["soft"]))
    o = {n: np.concatenate([g[n] for g in got]) for m in ("dx", "ddt", "dB", "dC") for n in (m, m + "|")}
    o.update({n: sum(g[n] for g in got) for m in ("dA", "dD", "ddt_bias") for n in (m, m + "|")})
    o.update({n: np.stack([g[n] for g in got]) for n in ("dh0", "dh0|")})
    return o


def run(c, lens=None, B=None, **kw):
    sh = (lambda t: t[None]) if B is None else (lambda t: t.unflatten(0, (B, -1)))
    return kda.ssm_bwd_chunked(sh(c["x"]), sh(c["dt"]), c["A"], sh(c["B"]), sh(c["C"]), sh(c["dy"]), c["h0"], c["dht"], D=c["D"],
                               dt_bias=c["bias"], softplus=c["soft"], cu_seqlens=None if B else cuts(lens), **kw)


def grads(c, lens, seed=5, dht=True):
    r = np.random.default_rng(seed)
    c["dy"] = cast(r.standard_normal(tuple(c["x"].shape)), c["x"].dtype).cuda()
    H, dv, dk = c["x"].shape[1], c["x"].shape[2], c["B"].shape[2]
    c["dht"] = cast(r.standard_normal((len(lens), H, dk, dv)), torch.float32).cuda() if dht else None
    return c


def compare(c, g, o, lens, dtype):
    k = 3 * (250 + 4 * (max(lens) // 64 + 1)) * U
    hb = 2.0 ** -8 * 1.01 if dtype == torch.bfloat16 else 0.0
    for n in NAMES:
        if n == "dh0" and c["h0"] is None or n == "dD" and c["D"] is None or n == "ddt_bias" and c["bias"] is None:
            assert g[n] is None
            continue
        want, size = o[n], o[n + "|"]
        got = g[n].reshape(want.shape)
        if n == "ddt":
            cu = cuts(lens)
            size = size.copy()
            for i, ln in enumerate(lens):
                if ln:
                    size[cu[i]:cu[i + 1]] = size[cu[i]:cu[i + 1]].max(0)
        tol = size * k * (4 if n in ("ddt", "dA", "ddt_bias") else 1) + (hb * size if n in ("dx", "dB", "dC") else 0)
        check(n, got, want, tol, g[n].dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens", [[1], [63], [64], [65], [5, 0, 1, 130, 64, 0], [600], [0, 2], [2] * 131, [3] * 130 + [800, 2]], ids=lambda l: f"{len(l)}x{sum(l)}")
@pytest.mark.parametrize("H,G,dk,dv,skip,soft,state,rows", [(2, 1, 64, 64, True, True, True, False), (4, 2, 128, 128, False, False, True, False),
                                                            (3, 3, 128, 64, True, True, False, True), (3, 1, 64, 128, True, True, True, True)])
def test_packed(dtype, lens, H, G, dk, dv, skip, soft, state, rows):
    say(f"ssm bwd packed {dtype} N={len(lens)} T={sum(lens)} H={H} G={G} dk={dk} dv={dv}")
    c = grads(make(lens, H, G, dk, dv, dtype, 41, skip, soft, state, rows), lens, dht=state)
    o = oracle(c, lens)
    g = run(c, lens)
    again = run(c, lens)
    torch.cuda.synchronize()
    compare(c, g, o, lens, dtype)
    for n in NAMES:
        assert g[n] is None or torch.equal(g[n], again[n]), n


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,T,H,G", [(2, 300, 8, 1), (1, 64, 12, 2), (9, 100, 2, 1), (2, 1300, 2, 1)])
def test_batch(dtype, B, T, H, G):
    say(f"ssm bwd batch {dtype} B={B} T={T} H={H} G={G}")
    lens = [T] * B
    c = grads(make(lens, H, G, 128, 128, dtype, 42, rate=2.0), lens)
    g = run(c, B=B)
    torch.cuda.synchronize()
    compare(c, g, oracle(c, lens), lens, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("name", ["x", "B", "C", "dt", "dy"])
def test_a_nan_token_stays_in_its_sequence_and_before_or_behind_its_chunk(dtype, name):
    # token 64 + 20 of the second sequence: x, B and dt reach later tokens, dy
    # (and C beside it) earlier ones; a whole chunk of 64 may become NaN
    say(f"ssm bwd bad token {dtype} {name}")
    lens = [100, 300, 30]
    c = grads(make(lens, 2, 1, 64, 64, dtype, 45, rate=2.0), lens, dht=False)
    want = run(c, lens)
    c[name][100 + 84] = float("nan")
    got = run(c, lens)
    for n in ("dx", "ddt", "dB", "dC"):
        a, b = got[n][0], want[n][0]
        assert torch.equal(a[:100], b[:100]) and torch.equal(a[400:], b[400:]), n
        if name in ("x", "B"):
            assert torch.equal(a[100:164], b[100:164]), n
        if name in ("dy", "C"):
            assert torch.equal(a[228:400], b[228:400]), n
    assert torch.equal(got["dh0"][0], want["dh0"][0]) and torch.equal(got["dh0"][2], want["dh0"][2])


@pytest.mark.parametrize("dtype", DTYPES)
def test_masked_tokens(dtype):
    # raw step sizes of -inf and of the type's lowest value: Softplus and its
    # slope are zero there, the tokens leave the states alone
    lens = [100, 90]
    c = grads(make(lens, 2, 1, 64, 64, dtype, 46, rate=2.0), lens)
    c["dt"][20:30] = float("-inf")
    c["dt"][95:110] = torch.finfo(dtype).min
    g = run(c, lens)
    torch.cuda.synchronize()
    compare(c, g, oracle(dict(c, dt=c["dt"].clamp(min=-1e3)), lens), lens, dtype)


def test_captured_and_replayed():
    lens = [300, 1, 0, 60]
    c = grads(make(lens, 2, 1, 64, 128, torch.bfloat16, 43), lens)
    ws = torch.empty(kda.lib().kda_ssm_bwd_workspace_bytes(1, 361, 2, 1, 64, 128, 1, 4), dtype=torch.uint8, device="cuda")
    out = {n: t.clone() for n, t in run(c, lens).items()}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run(c, lens, workspace=ws, out=out)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(c, lens, workspace=ws, out=out)
    for _ in range(3):
        c["dy"].normal_()
        ws.fill_(255)   # NaN bits: nothing of an earlier call is read
        g.replay()
        torch.cuda.synchronize()
        got = {n: t.clone() for n, t in out.items()}
        want = run(c, lens)
        torch.cuda.synchronize()
        for n in NAMES:
            assert torch.equal(got[n], want[n]), n


def test_gradient_by_differences_of_the_forward():
    # the library's own forward in fp32, along one direction of every input
    lens = [70, 40]
    c = grads(make(lens, 2, 1, 64, 64, torch.float32, 44, rate=2.0), lens)
    g = run(c, lens)
    r = np.random.default_rng(3)
    names = {"x": "dx", "dt": "ddt", "A": "dA", "B": "dB", "C": "dC", "D": "dD", "bias": "ddt_bias", "h0": "dh0"}
    step = 2.0 ** -7
    for n, gn in names.items():
        v = cast(r.standard_normal(tuple(c[n].shape)), torch.float32).cuda()

        def loss(sign):
            d = dict(c, **{n: c[n] + sign * step * v})
            y, ht = kda.ssm_fwd_chunked(d["x"][None], d["dt"][None], d["A"], d["B"][None], d["C"][None], d["h0"], D=d["D"], dt_bias=d["bias"],
                                        softplus=True, cu_seqlens=cuts(lens))
            return (f64(y[0]) * f64(c["dy"])).sum() + (f64(ht) * f64(c["dht"])).sum()
        want = (loss(1) - loss(-1)) / (2 * step)
        got = (f64(g[gn]).reshape(f64(v).shape) * f64(v)).sum()
        # the central difference's own error: step^2 / 6 of the third derivative, below 1e-2 of the sum of the products' sizes here
        size = np.abs(f64(g[gn]).reshape(f64(v).shape) * f64(v)).sum()
        assert abs(got - want) <= 1e-2 * size, (n, got, want, size)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("big", [2.0 ** 13, 2.0 ** 20])
def test_small_steps_behind_a_reset(dtype, big):
    from test_gpu_ssm import reset_case
    say(f"ssm bwd reset {dtype} dt={big}")
    c = grads(reset_case(dtype, big, False, 47), [200])
    g = run(c, [200])
    torch.cuda.synchronize()
    compare(c, g, oracle(c, [200]), [200], dtype)


@pytest.mark.parametrize("dtype", DTYPES)
def test_token_sums_that_cancel(dtype):
    # No decay (A = 0), steps of one, unit vectors as B and x: the products of a
    # chunk are R_ij = C_i[j] dy_i[j], whole numbers of our choice.  Large ones
    # cancel within rows and columns, and every sum is exact in 64 bits: dA =
    # sum_ij R_ij (i - j) and ddt_j = sum_i R_ij come out to their own rounding.
    say(f"ssm bwd cancelling sums {dtype}")
    n, big = 64, 2.0 ** 13
    r = np.random.default_rng(48)
    C, dy = r.integers(-2, 3, (n, n)).astype(float), np.ones((n, n))
    for i, j, s in ((20, 0, 1), (20, 8, -1), (28, 8, 1), (28, 0, -1), (45, 33, 1), (45, 38, -1), (47, 38, 1), (47, 33, -1), (60, 3, 1), (60, 40, -1),
                    (62, 40, 1), (62, 3, -1)):
        C[i, j], dy[i, j] = s * big, big
    C, dy = np.tril(C), np.tril(dy)
    one = lambda a: cast(a, dtype).cuda()
    v = lambda a: cast(a, torch.float32).cuda()
    e = np.eye(n)
    g = kda.ssm_bwd_chunked(one(e[None, :, None]), one(np.ones((1, n, 1))), v(np.zeros(1)), one(e[None, :, None]), one(C[None, :, None]),
                            one(dy[None, :, None]), dt_bias=v(np.zeros(1)))
    torch.cuda.synchronize()
    R, at = C * dy, np.arange(n)
    ddt = R.sum(0)
    check("dA", g["dA"], np.array([(R * (at[:, None] - at)).sum()]), 0.0, torch.float32)
    check("ddt_bias", g["ddt_bias"], np.array([ddt.sum()]), 0.0, torch.float32)
    check("ddt", g["ddt"][0, :, 0], ddt, 0.0, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
def test_small_steps_behind_a_reset_of_the_largest_step(dtype):
    from test_gpu_ssm import reset_case
    say(f"ssm bwd reset {dtype} dt=max")
    c = grads(reset_case(dtype, torch.finfo(dtype).max, False, 49), [200])
    g = run(c, [200])
    torch.cuda.synchronize()
    compare(c, g, oracle(c, [200]), [200], dtype)
