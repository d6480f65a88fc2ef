"""Places of the gated linear recurrence that its own tests do not reach.

Tolerances are those of test_gpu_lru.py where nothing else is said.
"""
import numpy as np
import pytest
import torch

import test_gpu_lru as tl
from gated_delta_rule_96_amd import kda
from kda_testutil import say

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
DTYPES = [F32, BF]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens,top", [([12, 5], 3.0), ([300], 0.15)], ids=str)
def test_log_decays_above_zero_are_computed_as_they_are(dtype, lens, top):
    say(f"recurrence {dtype} {lens} log-decays to {top}")
    for D in (130, 7):
        k = tl.make(lens, D, dtype, 201 + D, gate=False)
        r = np.random.default_rng(202)
        g = r.uniform(-top, top, (1, sum(lens), D))
        g[0, 0], g[0, 3], g[0, 4] = top / 3, top, 0.0
        k["r"] = tl.dev(g, dtype)
        kw = dict(unit=False, cu_seqlens=tl.cuts(lens))
        y, ht = kda.lru_fwd(k["x"], k["r"], k["i"], None, k["h0"], **kw)
        gr = kda.lru_bwd(k["x"], k["r"], k["i"], None, k["dy"], k["h0"], k["dht"], **kw)
        state = k["h0"][:1].clone()
        steps = [kda.lru_step(k["x"][:, t], k["r"][:, t], k["i"][:, t], None, state, unit=False) for t in range(5)]
        m, _ = kda.lru_fwd(k["x"], k["r"], k["i"], None, k["h0"], cu_seqlens=tl.cuts(lens))
        torch.cuda.synchronize()
        want = tl.oracle(k, lens, False, back=True)
        tl.check("y", y[0], want["y"], want["ty"], dtype)
        tl.check("ht", ht, want["ht"], want["tht"], F32)
        tl.check("steps", torch.cat(steps), want["y"][:5], want["ty"][:5], dtype)
        tl.compare_grads(k, gr, want, dtype)
        assert torch.isnan(m[0, 0]).all()   # (its root of 1 - a^2)


def test_dc_of_more_channels_than_one_launch_sums():
    # a column sum of 64 channels a work-group of 1024: one launch has them for
    # 64 (2^22 - 1) channels.  Channels are on their own, so halves have the same bits.
    B, D = 2, (1 << 28) + 128
    say(f"recurrence gradients {B} x 1 x {D}")
    gen = torch.Generator(device="cuda").manual_seed(271)
    x = torch.randn((B, 1, D), dtype=BF, device="cuda", generator=gen)
    c = torch.rand(D, device="cuda", generator=gen)
    h0 = torch.full((B, D), 0.5, device="cuda")
    dc = torch.full((D,), float("nan"), device="cuda")
    got = kda.lru_bwd(x, x, None, c, x, h0, out=dict(dx=torch.empty_like(x), dr=torch.empty_like(x), di=None, dc=dc, dh0=None))
    for lo in (0, D // 2):
        part, at = x[..., lo:lo + D // 2].contiguous(), slice(lo, lo + D // 2)
        half = kda.lru_bwd(part, part, None, c[at].clone(), part, h0[:, at].contiguous())
        torch.cuda.synchronize()
        assert torch.equal(dc[at], half["dc"]) and torch.equal(got["dr"][..., at], half["dr"])
        del half, part
    assert float(dc.abs().min()) >= 0 and int((dc != 0).sum()) > 0.9 * D
    del got, x, c, h0, dc
    torch.cuda.empty_cache()


def test_gradients_of_more_chains_than_one_launch_carries():
    # 131072 sequences of two parts: 33 work-groups of 64 channels each, over 2^22
    # together.  256 sequences over and over, so every repetition has their bits.
    B, T, D, few = 1 << 17, 33, 2056, 256
    say(f"recurrence gradients {B} x {T} x {D}")
    torch.cuda.empty_cache()
    gen = torch.Generator(device="cuda").manual_seed(281)
    part = torch.randn((few, T, D), dtype=BF, device="cuda", generator=gen)
    c = torch.rand(D, device="cuda", generator=gen)
    want = kda.lru_bwd(part, part, None, c, part)
    x = torch.empty((B, T, D), dtype=BF, device="cuda")
    x.view(B // few, few, T, D).copy_(part)
    got = kda.lru_bwd(x, x, None, c, x)
    torch.cuda.synchronize()
    for n in ("dx", "dr"):
        all_of = got[n].view(B // few, few, T, D)
        assert all(torch.equal(all_of[k], want[n]) for k in range(B // few)), n
    # (dc: the same terms B / few times, joined in 64 bits and rounded once on each side)
    torch.testing.assert_close(got["dc"].double(), want["dc"].double() * (B // few), rtol=2.0 ** -22, atol=0)
    del x, got, all_of
    torch.cuda.empty_cache()


def test_gradients_of_the_recurrence_along_themselves():
    # Every leaf along its own gradient G, d = G / max |G|: the slope is sum G^2 /
    # max |G|, which no wrong sign, place or factor gives.  The forward's central
    # difference on the GPU has the error of its two values (the forward's
    # tolerance, and half a unit of y, weighted by |dy|, over 2 e), and that of the step itself,
    # which the oracle's difference of the same inputs has too.
    lens = [40]
    k = tl.make(lens, 16, F32, 211)
    want = tl.oracle(k, lens, True, back=True)
    g = kda.lru_bwd(k["x"], k["r"], k["i"], k["c"], k["dy"], k["h0"], k["dht"])
    e = 2.0 ** -6
    for n in ("x", "r", "i", "c", "h0"):
        G, tol = want["d" + n], want["td" + n]
        d = tl.dev((G / np.abs(G).max()).reshape(k[n].shape))

        def sides(s):
            v = dict(k, **{n: k[n] + s * d})
            y, ht = kda.lru_fwd(v["x"], v["r"], v["i"], v["c"], v["h0"])
            o = tl.oracle(v, lens, True)
            f = lambda y, ht: float((y * tl.f64(k["dy"])[0]).sum() + (ht * tl.f64(k["dht"])).sum())
            err = float(((o["ty"] + U * np.abs(o["y"])) * np.abs(tl.f64(k["dy"])[0])).sum() + (o["tht"] * np.abs(tl.f64(k["dht"]))).sum())
            return f(tl.f64(y[0]), tl.f64(ht)), f(o["y"], o["ht"]), err
        (a, a64, ea), (b, b64, eb) = sides(e), sides(-e)
        d64 = tl.f64(d).reshape(G.shape)
        slope, slope64, exact = (a - b) / (2 * e), (a64 - b64) / (2 * e), float((G * d64).sum())
        lim = (ea + eb) / (2 * e)
        step = abs(slope64 - exact)
        grad = float(((tol + U * np.abs(G)) * np.abs(d64)).sum())
        got = float((tl.f64(g["d" + n]).reshape(G.shape) * d64).sum())
        assert lim + step + grad <= 0.1 * exact, (n, lim, step, grad, exact)
        assert abs(slope - slope64) <= lim and abs(got - exact) <= grad and abs(got - slope) <= lim + step + grad, n


@pytest.mark.parametrize("dtype", DTYPES)
def test_states_that_start_on_four_bytes(dtype):
    # pairs of channels fit the rows but not the states
    D, T, B = 34, 300, 3
    k = tl.make([T] * B, D, dtype, 261)
    rows = [k[n].reshape(B, T, D) for n in ("x", "r", "i")]
    odd = lambda: torch.full((B * D + 8,), 5.0, device="cuda")
    want, wht = kda.lru_fwd(*rows, k["c"], k["h0"])
    gw = kda.lru_bwd(*rows, k["c"], k["dy"].reshape(B, T, D), k["h0"], k["dht"])
    for src, dst in ((1, 0), (0, 1), (1, 1)):
        a, b = odd(), odd()
        h0, ht = a[src:src + B * D].view(B, D), b[dst:dst + B * D].view(B, D)
        h0.copy_(k["h0"])
        y, _ = kda.lru_fwd(*rows, k["c"], h0, ht=ht)
        assert torch.equal(y, want) and torch.equal(ht, wht) and bool((b[:dst] == 5).all()) and bool((b[dst + B * D:] == 5).all())
        ht.copy_(h0)
        y = kda.lru_step(*(t[:, 0] for t in rows), k["c"], ht)
        so = torch.empty((B, D), device="cuda")
        y2 = kda.lru_step(*(t[:, 0].contiguous() for t in rows), k["c"], k["h0"], state_out=so)
        assert torch.equal(y, y2) and torch.equal(ht, so) and torch.equal(y2, want[:, 0]) and bool((b[dst + B * D:] == 5).all())
        dht, dh0 = odd()[src:src + B * D].view(B, D), b[dst:dst + B * D].view(B, D)
        dht.copy_(k["dht"])
        g = kda.lru_bwd(*rows, k["c"], k["dy"].reshape(B, T, D), h0, dht, out=dict(gw, dh0=dh0, dx=torch.empty_like(gw["dx"])))
        assert torch.equal(g["dx"], gw["dx"]) and torch.equal(dh0, kda.lru_bwd(*rows, k["c"], k["dy"].reshape(B, T, D), k["h0"], k["dht"])["dh0"])


@pytest.mark.parametrize("lens,D", [([100], 64), ([700], 64), ([700], 2048), ([128] * 200, 40), ([5] * 130 + [900], 40), ([900] + [5] * 200, 2048)], ids=lambda v: str(v)[:24])
def test_status_word_of_the_workspace(lens, D):
    # every schedule (sequences of one part; parts that look back far and near;
    # several launches) clears what was there, and a sound call leaves it clear
    k = tl.make(lens, D, BF, 301)
    ws = torch.full((kda.lib().kda_lru_workspace_bytes(1, sum(lens), D, len(lens)),), 255, dtype=torch.uint8, device="cuda")
    assert kda.workspace_error(ws) == kda.KDA_ERR_INCOMPLETE
    kda.lru_fwd(k["x"], k["r"], k["i"], k["c"], k["h0"], cu_seqlens=tl.cuts(lens), workspace=ws)
    kda.check_workspace(ws)
    assert kda.workspace_error(ws) == 0
