"""Workloads of the operators a recurrent block adds around its sequence mixer:
the root-mean-square norm of the residual stream with the residual's addition
(outputs of the stream's type, or in 8 bits with a scale for every 128
channels; gradients), the product of such 8-bit rows with 8-bit weights, and
the gated linear recurrence of one state a channel (prompts, packed prompts,
single tokens, gradients).

Each case can run in two forms on the same inputs: a plain one in elementary
torch operations (32-bit arithmetic, one rounding at the end), and, with `own`
set, the library's calls.  `exact` gives the operators' definitions in 64 bits.
"""
import math
import random

import torch
import torch.nn.functional as F

own = False

DEVICE = "cuda"
Q = 64          # tokens per chunk of the plain recurrence
BLOCK = 128     # channels that share a scale
E4M3 = 448.0    # largest value of the 8-bit type
EPS = 1e-6
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- the cases
def listed():
    """Every case names what it stands for in a model's step."""
    return [
        # residual stream of a 64K prompt into the 8-bit input of the projections (32 heads of 128 channels)
        dict(name="norm 64K prompt to 8 bits", op="norm_fwd", dtype="bf16", res="bf16", rows=65536, D=4096, fp8=True, weight=True, pad=0),
        # one token for each of 256 sequences
        dict(name="norm token B256 to 8 bits", op="norm_fwd", dtype="bf16", res="bf16", rows=256, D=4096, fp8=True, weight=True, pad=0),
        # packed prompts with the stream kept in 32 bits, the addend a slice of a wider tensor, a width that is no power of two
        dict(name="norm packed, 32-bit stream", op="norm_fwd", dtype="bf16", res="f32", rows=8191, D=2056, fp8=False, weight=True, pad=72),
        # a training batch's gradients, with the residual path's own
        dict(name="norm gradients", op="norm_bwd", dtype="bf16", dy="bf16", rows=32768, D=4096, weight=True, skip=True),
        # projection of a long prompt's rows to queries, keys and values of 32 heads
        dict(name="product 8K prompt", op="product", M=8192, N=12288, K=4096, out="bf16"),
        # packed prompts to the rows the convolution and the scan cut into slices
        dict(name="product packed prompts", op="product", M=8191, N=8480, K=4096, out="bf16"),
        # one token for each of 256 sequences
        dict(name="product token B256", op="product", M=256, N=12288, K=4096, out="bf16"),
        # a single token, output in 32 bits
        dict(name="product one token", op="product", M=1, N=12288, K=4096, out="f32"),
        # a 64K prompt through the recurrence
        dict(name="recurrence 64K prompt", op="lru_fwd", dtype="bf16", B=1, T=65536, D=4096, N=0, cut=0, pad=0, gate=True, igate=True, unit=True, state=True),
        # packed prompts in 32 bits, gates and inputs as slices of one projection
        dict(name="recurrence packed prompts f32", op="lru_fwd", dtype="f32", B=1, T=8191, D=4096, N=11, cut=5, pad=8, gate=True, igate=True, unit=True, state=True),
        # one token for each of 256 sequences
        dict(name="recurrence token B256", op="lru_step", dtype="bf16", B=256, T=1, D=4096, N=0, cut=0, pad=0, gate=True, igate=True, unit=True, state=True),
        # a training batch's gradients
        dict(name="recurrence gradients", op="lru_bwd", dtype="bf16", B=4, T=8192, D=2048, N=0, cut=0, pad=0, gate=True, igate=True, unit=True, state=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_fwd", "norm_bwd", "product", "product", "product", "lru_fwd", "lru_fwd", "lru_step", "lru_bwd"])
    c = dict(op=op)
    if op.startswith("norm"):
        D = 8 * _log(rng, 1, 1024)
        lim = 1 << (27 if op == "norm_bwd" else 28)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        rows = max(1, min(_log(rng, 1, 65536), lim // (2 if dtype == "f32" else 1) // D))
        c.update(dtype=dtype, rows=rows, D=D, weight=rng.random() < 0.8)
        if op == "norm_fwd":
            c.update(res=rng.choice(["", "bf16", "f32"]) if dtype == "bf16" else rng.choice(["", "f32"]), fp8=rng.random() < 0.6, pad=rng.choice([0, 0, 8, 72]))
            if c["res"] == "f32":
                c["rows"] = max(1, min(rows, (lim >> 1) // D))
        else:
            c.update(dy=rng.choice(["bf16", "f32"]), skip=rng.random() < 0.7)
    elif op == "product":
        M, K = _log(rng, 1, 65536), 16 * _log(rng, 1, 1024)
        N = _log(rng, 1, 16384) if rng.random() < 0.4 else 64 * _log(rng, 1, 256)
        M = max(1, min(M, (1 << 27) // N, (1 << 28) // K, 8192 * 12288 * 4096 // (N * K)))
        c.update(M=M, N=N, K=K, out=rng.choice(["bf16", "bf16", "f32"]))
    else:
        dtype = rng.choice(["bf16", "bf16", "f32"])
        D = _log(rng, 3, 8192) if rng.random() < 0.4 else 64 * _log(rng, 1, 128)
        if op == "lru_step":
            B, T, N = _log(rng, 1, 1024), 1, 0
        else:
            T = _log(rng, 1, 65536)
            N = rng.choice([0, 0, _log(rng, 1, 200)])
            B = 1 if N else _log(rng, 1, 64)
            lim = (1 << 28) // (2 if dtype == "f32" else 1) // (8 if op == "lru_bwd" else 1)
            T = max(1, min(T, lim // (B * D)))
            N = min(N, T)
        gate = rng.random() < 0.8
        c.update(dtype=dtype, B=B, T=T, D=D, N=N, cut=rng.randrange(1000), pad=rng.choice([0, 0, 8, 13]), gate=gate, igate=rng.random() < 0.7,
                 unit=rng.random() < 0.7, state=rng.random() < 0.7)
    return c


def _lens(c):
    """Lengths of a case's sequences: B of T tokens, or N ragged ones of T in all."""
    if not c["N"]:
        return [c["T"]] * c["B"]
    r = random.Random(c["cut"])
    cuts = sorted(r.randrange(c["T"] + 1) for _ in range(c["N"] - 1))
    ends = [0] + cuts + [c["T"]]
    return [ends[i + 1] - ends[i] for i in range(c["N"])]


# ---------------------------------------------------------------- inputs
def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _scale(amax):
    return torch.where(amax > 0, amax / E4M3, torch.ones_like(amax))


def _row_scales(x):
    """Scales [rows, blocks] of 32-bit rows, one for every 128 channels."""
    n = x.shape[-1]
    return _scale(F.pad(x.abs(), (0, _blocks(n) * BLOCK - n)).unflatten(-1, (-1, BLOCK)).amax(-1))


def _spread(s, n):
    """[..., blocks] -> [..., n]: every channel its block's scale."""
    return s.repeat_interleave(BLOCK, -1)[..., :n]


def prepare(c, seed):
    dev = DEVICE
    gen = torch.Generator(device=dev).manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen, device=dev)
    ru = lambda *s: torch.rand(s, generator=gen, device=dev)
    # rows of a wider tensor where the case has padding (a slice of a projection's output)
    rows = lambda x, dt, pad: F.pad(x, (0, pad)).to(dt)[..., :x.shape[-1]]
    s = {"c": c}
    if c["op"].startswith("norm"):
        R, D, dt = c["rows"], c["D"], DT[c["dtype"]]
        size = torch.exp(0.5 * rn(D))   # channels of unlike size, as a trained stream has them
        s["w"] = 1 + 0.2 * rn(D) if c["weight"] else None
        if c["op"] == "norm_fwd":
            s["x"] = rows(rn(R, D) * size, dt, c["pad"])
            s["res"] = (2.0 * rn(R, D) * size).to(DT[c["res"]]) if c["res"] else None
        else:
            s["h"] = (2.0 * rn(R, D) * size).to(dt)
            s["dy"] = rn(R, D).to(DT[c["dy"]])
            s["dh"] = rn(R, D).to(dt) if c["skip"] else None
    elif c["op"] == "product":
        M, N, K = c["M"], c["N"], c["K"]
        x = rn(M, K) * torch.exp(0.5 * rn(K))
        s["sa"] = _row_scales(x)
        s["a"] = (x / _spread(s["sa"], K)).to(torch.float8_e4m3fn)
        w = rn(N, K) / math.sqrt(K)
        tiles = F.pad(w.abs(), (0, _blocks(K) * BLOCK - K, 0, _blocks(N) * BLOCK - N)).unflatten(1, (-1, BLOCK)).unflatten(0, (-1, BLOCK))
        s["sw"] = _scale(tiles.amax((1, 3)))
        s["w"] = (w / _spread(s["sw"], K).repeat_interleave(BLOCK, 0)[:N]).to(torch.float8_e4m3fn)
    else:
        B, T, D, dt = c["B"], c["T"], c["D"], DT[c["dtype"]]
        lens = _lens(c)
        N = len(lens)
        # decays of 0.9 to 0.999 a token where the gate is open
        s["cc"] = -torch.log(0.9 + 0.099 * ru(D)) if c["gate"] else None
        s["x"] = rows(rn(B, T, D), dt, c["pad"])
        s["r"] = rows(rn(B, T, D) if c["gate"] else torch.log(0.9 + 0.099 * ru(B, T, D)), dt, c["pad"])
        s["i"] = rows(rn(B, T, D), dt, c["pad"]) if c["igate"] else None
        s["h0"] = rn(N, D) if c["state"] else None
        if c["op"] == "lru_step":
            s["x"], s["r"] = s["x"][:, 0], s["r"][:, 0]
            s["i"] = s["i"][:, 0] if c["igate"] else None
            s["h0"] = rn(N, D)
            s["state"] = torch.empty_like(s["h0"])
        if c["op"] == "lru_bwd":
            s["dy"] = rn(B, T, D).to(dt)
            s["dht"] = rn(N, D) if c["state"] else None
        s["cu"] = [sum(lens[:k]) for k in range(N + 1)] if c["N"] else None
        # the plain recurrence's layout: every sequence on chunks of its own, at least one
        ln = torch.tensor(lens)
        nch = ((ln + Q - 1) // Q).clamp(min=1)
        first = torch.cumsum(nch, 0) - nch
        cseq = torch.repeat_interleave(torch.arange(N), nch)
        within = torch.arange(int(nch.sum())) - first[cseq]
        start = torch.cumsum(ln, 0) - ln
        at = within[:, None] * Q + torch.arange(Q)
        tok = torch.where(at < ln[cseq][:, None], start[cseq][:, None] + at, B * T)
        s["plan"] = dict(tok=tok.to(dev), first=first.to(dev), last=(first + nch - 1).to(dev))
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    c = s["c"]
    if own:
        return _library(s, c)
    return {"norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd, "product": _product, "lru_fwd": _lru_fwd, "lru_step": _lru_step, "lru_bwd": _lru_bwd}[c["op"]](s, c)


def _library(s, c):
    from gated_delta_rule_96_amd import kda
    op = c["op"]
    if op == "norm_fwd":
        y, h = kda.add_rms_norm(s["x"], s["res"], s["w"], eps=EPS, fp8=c["fp8"])
        return {"y": y[0] if c["fp8"] else y, "scale": y[1] if c["fp8"] else None, "h": h}
    if op == "norm_bwd":
        return kda.add_rms_norm_bwd(s["h"], s["w"], s["dy"], s["dh"], eps=EPS)
    if op == "product":
        return kda.gemm_fp8(s["a"], s["sa"], s["w"], s["sw"], out_dtype=DT[c["out"]])
    if op == "lru_fwd":
        return kda.lru_fwd(s["x"], s["r"], s["i"], s["cc"], s["h0"], unit=c["unit"], cu_seqlens=s["cu"])
    if op == "lru_step":
        return kda.lru_step(s["x"], s["r"], s["i"], s["cc"], s["h0"], unit=c["unit"], state_out=s["state"]), s["state"]
    return kda.lru_bwd(s["x"], s["r"], s["i"], s["cc"], s["dy"], s["h0"], s["dht"], unit=c["unit"], cu_seqlens=s["cu"])


# ---------------------------------------------------------------- norm of the residual stream
# h = x + res, rounded to the stream's type; n = w h / sqrt(mean h^2 + eps)
def _norm_fwd(s, c):
    h = s["x"]
    if s["res"] is not None:
        h = (s["x"].float() + s["res"].float()).to(s["res"].dtype)
    f = h.float()
    n = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS)
    n = n * s["w"] if s["w"] is not None else n
    scale = _row_scales(n) if c["fp8"] else None
    y = (n / _spread(scale, c["D"])).to(torch.float8_e4m3fn) if c["fp8"] else n.to(s["x"].dtype)
    return {"y": y, "scale": scale, "h": h if s["res"] is not None else None}


def _norm_bwd(s, c):
    f, g = s["h"].float(), s["dy"].float()
    r = torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS)
    u = f * r
    dw = (g * u).sum(0, dtype=torch.float64).float() if s["w"] is not None else None
    g = g * s["w"] if s["w"] is not None else g
    dx = r * (g - u * (g * u).mean(-1, keepdim=True))
    dx = dx + s["dh"].float() if s["dh"] is not None else dx
    return {"dx": dx.to(s["h"].dtype), "dw": dw}


# ---------------------------------------------------------------- product of 8-bit rows and weights
def _product(s, c):
    a = s["a"].float() * _spread(s["sa"], c["K"])
    w = s["w"].float() * _spread(s["sw"], c["K"]).repeat_interleave(BLOCK, 0)[:c["N"]]
    return torch.matmul(a, w.t()).to(DT[c["out"]])


# ---------------------------------------------------------------- the gated linear recurrence
# g_t = -c Sigmoid(r_t) (or r_t itself), a_t = e^g_t, h_t = a_t h_{t-1} + m_t Sigmoid(i_t) x_t, m_t = sqrt(1 - a_t^2) (or 1)
def _parts(s, c, x, r, i):
    """g, a, m and the input gate of 32-bit rows."""
    g = -s["cc"] * torch.sigmoid(r) if c["gate"] else r
    m = torch.sqrt(-torch.expm1(2 * g)) if c["unit"] else torch.ones_like(g)
    return g, torch.exp(g), m, torch.sigmoid(i) if c["igate"] else torch.ones_like(x)


def _leaves(s, c):
    f = lambda n: s[n].float() if s[n] is not None else None
    return f("x"), f("r"), f("i")


def _scan(a, u, head, start):
    """h_t = a_t h_{t-1} + u_t over chunks [nc, Q, D]; the chunks listed in `head` begin with the state `start`."""
    h, p = torch.empty_like(u), torch.empty_like(a)
    h[:, 0], p[:, 0] = u[:, 0], a[:, 0]
    for t in range(1, Q):
        torch.addcmul(u[:, t], a[:, t], h[:, t - 1], out=h[:, t])
        torch.mul(a[:, t], p[:, t - 1], out=p[:, t])
    # state entering every chunk: the same recurrence over chunks, by doubling
    A, U = p[:, -1].clone(), h[:, -1].clone()
    U[head] += A[head] * start
    A[head] = 0
    d = 1
    while d < A.shape[0]:
        U[d:] = U[d:] + A[d:] * U[:-d]
        A[d:] = A[d:] * A[:-d]
        d *= 2
    enter = torch.cat([torch.zeros_like(U[:1]), U[:-1]])
    enter[head] = start
    return h + p * enter[:, None], enter, U


def _chunks(v, s, fill):
    """Rows [B, T, D] as [nc, Q, D]; `fill` behind a sequence's last."""
    v = v.reshape(-1, v.shape[-1])
    return torch.cat([v, torch.full_like(v[:1], fill)])[s["plan"]["tok"]]


def _rows(v, s, c):
    """Chunks back to rows [B, T, D]."""
    out = v.new_empty(c["B"] * c["T"] + 1, c["D"])
    out[s["plan"]["tok"].reshape(-1)] = v.reshape(-1, c["D"])
    return out[:-1].view(c["B"], c["T"], c["D"])


def _start(s, c):
    return s["h0"] if s["h0"] is not None else torch.zeros(s["plan"]["first"].shape[0], c["D"], device=s["x"].device)


def _lru_fwd(s, c):
    x, r, i = _leaves(s, c)
    _, a, m, si = _parts(s, c, x, r, i)
    h, _, U = _scan(_chunks(a, s, 1.0), _chunks(m * si * x, s, 0.0), s["plan"]["first"], _start(s, c))
    return _rows(h, s, c).to(s["x"].dtype), U[s["plan"]["last"]]


def _lru_step(s, c):
    x, r, i = _leaves(s, c)
    _, a, m, si = _parts(s, c, x, r, i)
    h = a * s["h0"] + m * si * x
    s["state"].copy_(h)
    return h.to(s["x"].dtype), s["state"]


def _lru_bwd(s, c):
    x, r, i = _leaves(s, c)
    g, a, m, si = _parts(s, c, x, r, i)
    p, dt = s["plan"], s["x"].dtype
    ac = _chunks(a, s, 1.0)
    h, enter, _ = _scan(ac, _chunks(m * si * x, s, 0.0), p["first"], _start(s, c))
    before = _rows(torch.cat([enter[:, None], h[:, :-1]], 1), s, c)      # h_{t-1}
    # dL/dh_t = dy_t + a_{t+1} dL/dh_{t+1}: e_t = a_t (dy_t + e_{t+1}) backwards
    dyc = _chunks(s["dy"].float(), s, 0.0)
    tail = s["dht"] if s["dht"] is not None else torch.zeros(p["last"].shape[0], c["D"], device=x.device)
    back = lambda v: v.flip(0, 1)
    e, enter, U = _scan(back(ac), back(ac * dyc), ac.shape[0] - 1 - p["last"], tail)
    dh0 = U[ac.shape[0] - 1 - p["first"]]
    lam = _rows(back(torch.cat([enter[:, None], e[:, :-1]], 1)) + dyc, s, c)
    dm = lam * si * x
    pull = lam * before * a                                                # through the decay
    out = {"dx": (lam * m * si).to(dt)}
    if c["gate"]:
        sr = torch.sigmoid(r)
        if c["unit"]:
            pull = pull - dm * a * a / m
        out["dr"] = (pull * g * (1 - sr)).to(dt)
        out["di"] = None
        out["dc"] = -(pull * sr).sum((0, 1), dtype=torch.float64).float()
    else:
        out["dr"] = (pull - dm * a * a / m if c["unit"] else pull).to(dt)
        out["di"] = out["dc"] = None
    if c["igate"]:
        out["di"] = (lam * m * x * si * (1 - si)).to(dt)
    out["dh0"] = dh0 if s["h0"] is not None else None
    return out


# ---------------------------------------------------------------- cost
def work(c):
    e = lambda t: {"bf16": 2, "f32": 4, "": 0}[t]
    op = c["op"]
    if op == "norm_fwd":
        n, D = c["rows"] * c["D"], c["D"]
        out = n + 4 * c["rows"] * _blocks(D) if c["fp8"] else n * e(c["dtype"])
        return {"bytes": n * (e(c["dtype"]) + 2 * e(c["res"])) + out + (4 * D if c["weight"] else 0), "flops": n * (8 if c["fp8"] else 5)}
    if op == "norm_bwd":
        n = c["rows"] * c["D"]
        return {"bytes": n * (e(c["dtype"]) * (3 if c["skip"] else 2) + e(c["dy"])) + (8 * c["D"] if c["weight"] else 0), "flops": n * 11}
    if op == "product":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": M * K + N * K + 4 * _blocks(K) * (M + _blocks(N)) + M * N * e(c["out"]), "flops": 2 * M * N * K}
    n, D, z = c["B"] * c["T"] * c["D"], c["D"], e(c["dtype"])
    ins = 2 + c["igate"]
    st = (c["N"] or c["B"]) * D * 4
    gates = 6 * (c["gate"] + c["igate"]) + 4 * c["unit"]
    if op == "lru_bwd":
        return {"bytes": n * z * (2 * ins + 1) + (3 if c["state"] else 0) * st + 8 * D, "flops": n * (20 + 2 * gates)}
    return {"bytes": n * z * (ins + 1) + (1 + bool(c["state"])) * st + 4 * D, "flops": n * (5 + gates)}


# ---------------------------------------------------------------- definitions in 64 bits
def exact(c, seed):
    s = prepare(c, seed)
    d = lambda n: s[n].double() if s.get(n) is not None else None
    if c["op"] == "product":
        cut = lambda v, b: torch.arange(v, device=DEVICE) // b
        a = d("a") * d("sa")[:, cut(c["K"], BLOCK)]
        w = d("w") * d("sw")[cut(c["N"], BLOCK)][:, cut(c["K"], BLOCK)]
        return a @ w.t()
    if c["op"].startswith("norm"):
        return _exact_norm(s, c, d)
    return _exact_lru(s, c, d)


def _exact_norm(s, c, d):
    R, D = c["rows"], c["D"]
    w = d("w") if s["w"] is not None else torch.ones(D, dtype=torch.float64, device=DEVICE)
    per = max(1, (1 << 25) // D)
    got = {"y": [], "scale": [], "h": [], "dx": []}
    dw = torch.zeros(D, dtype=torch.float64, device=DEVICE)
    for lo in range(0, R, per):
        at = slice(lo, lo + per)
        if c["op"] == "norm_bwd":
            h, g = s["h"][at].double(), s["dy"][at].double()
            rms = (h.square().sum(1, keepdim=True) / D + EPS).sqrt()
            dw += (g * h / rms).sum(0)
            g = g * w
            dx = g / rms - h * (g * h).sum(1, keepdim=True) / (D * rms ** 3)
            got["dx"].append(dx + s["dh"][at].double() if s["dh"] is not None else dx)
            continue
        h = s["x"][at].double()
        if s["res"] is not None:
            h = (h + s["res"][at].double()).to(s["res"].dtype).double()
            got["h"].append(h)
        y = w * h / (h.square().sum(1, keepdim=True) / D + EPS).sqrt()
        if c["fp8"]:
            top = torch.stack([b.abs().amax(1) for b in y.split(BLOCK, 1)], 1) / E4M3
            top[top == 0] = 1
            got["scale"].append(top)
            y = torch.cat([b / top[:, k:k + 1] for k, b in enumerate(y.split(BLOCK, 1))], 1)
        got["y"].append(y)
    cat = lambda n: torch.cat(got[n]) if got[n] else None
    if c["op"] == "norm_bwd":
        return {"dx": cat("dx"), "dw": dw if s["w"] is not None else None}
    return {"y": cat("y"), "scale": cat("scale"), "h": cat("h")}


def _exact_lru(s, c, d):
    """Token by token."""
    step = c["op"] == "lru_step"
    one = lambda v: v[:, None] if step else v
    x, r = one(d("x")), one(d("r"))
    sr = 1 / (1 + torch.exp(-r))
    g = -d("cc") * sr if c["gate"] else r
    a = g.exp()
    m = (-torch.expm1(2 * g)).sqrt() if c["unit"] else torch.ones_like(g)
    si = 1 / (1 + torch.exp(-one(d("i")))) if c["igate"] else torch.ones_like(x)
    u = m * si * x
    cuts = [(0, x.shape[1])] if s["cu"] is None else list(zip(s["cu"], s["cu"][1:]))
    n = x.shape[0] if s["cu"] is None else len(cuts)
    h0 = d("h0") if s["h0"] is not None else x.new_zeros(n, c["D"])
    own_rows = lambda v, k: v if s["cu"] is None else v[k:k + 1]   # states of the batch, or of sequence k
    y, fin = torch.empty_like(x), []
    before = torch.empty_like(x) if c["op"] == "lru_bwd" else None
    for k, (lo, hi) in enumerate(cuts):
        h = own_rows(h0, k)
        for t in range(lo, hi):
            if before is not None:
                before[:, t] = h
            h = torch.addcmul(u[:, t], a[:, t], h)
            y[:, t] = h
        fin.append(h)
    if c["op"] == "lru_step":
        return [y[:, 0], torch.cat(fin)]
    if c["op"] == "lru_fwd":
        return [y, torch.cat(fin)]
    lam, dh0, dy = y, [], d("dy")
    for k, (lo, hi) in enumerate(cuts):
        e = own_rows(d("dht"), k) if s["dht"] is not None else torch.zeros_like(own_rows(h0, k))
        for t in range(hi - 1, lo - 1, -1):
            lam[:, t] = dy[:, t] + e
            e = a[:, t] * lam[:, t]
        dh0.append(e)
    dg = lam * before * a
    if c["unit"]:
        dg = dg - lam * si * x * a.square() / m
    dr = dg * (-d("cc")) * sr * (1 - sr) if c["gate"] else dg
    return {"dx": lam * m * si, "dr": dr, "di": lam * m * x * si * (1 - si) if c["igate"] else None,
            "dc": (dg * -sr).sum((0, 1)) if c["gate"] else None, "dh0": torch.cat(dh0) if s["h0"] is not None else None}
