"""GPU parity of the product of 8-bit rows and weights (kda_gemm_fp8) against
the fp64 oracle (oracle/block.py).

Tolerances, per element, S = sum over blocks of |sa sw| sqrt(sum (a w)^2), u =
2^-24.  fp32 output: e4m3 products are exact in fp16 operands; 128 of them are
summed in fp32 (at most 128 u of their absolute sum A), KB blocks join with two
roundings of the scale and one of the fma: (131 + KB) u A with A = sum |sa sw| sum
|a w|.  bf16 output: the 8-bit matrix instruction rounds its products at a place
that their largest sets: of 2^20 random sums none was off by more than 6e-5 of
its sqrt(sum (a w)^2), bounded here by 2^-12 of it, and by h |c| for the rounding.
"""
import numpy as np
import pytest
import torch

from gated_delta_rule_96_amd import kda
from kda_testutil import cast, say
from oracle import block

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
F8, BF, F32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32


def f64(t):
    return t.detach().cpu().float().double().numpy()


def make(M, N, K, seed, pad=0):
    r = np.random.default_rng(seed)
    kb, nb = (K + 127) // 128, (N + 127) // 128
    wide = torch.full((M, K + pad), float("nan"), device="cuda").to(F8)
    wide[:, :K] = cast(np.clip(100 * r.standard_normal((M, K)) * np.exp(r.standard_normal((M, 1))), -448, 448), F32).to(F8).cuda()
    sa = torch.full((M, kb + (3 if pad else 0)), float("nan"), device="cuda")
    sa[:, :kb] = cast(np.exp(r.standard_normal((M, kb))), F32).cuda()
    w = cast(np.clip(100 * r.standard_normal((N, K)), -448, 448), F32).to(F8).cuda()
    return wide[:, :K], sa[:, :kb], w, cast(np.exp(r.standard_normal((nb, kb))), F32).cuda()


def check(a, sa, w, sw, c):
    A, SA, W, SW = (f64(t) for t in (a, sa, w, sw))
    M, K = A.shape
    N = W.shape[0]
    want, size, root = np.zeros((M, N)), np.zeros((M, N)), np.zeros((M, N))
    for k in range(0, K, 128):
        s = np.abs(SA[:, k // 128][:, None] * block.spread(SW[:, k // 128], N)[None])
        x, y = A[:, k:k + 128], W[:, k:k + 128]
        want += SA[:, k // 128][:, None] * block.spread(SW[:, k // 128], N)[None] * (x @ y.T)
        size += s * (np.abs(x) @ np.abs(y).T)
        root += s * np.sqrt((x * x) @ (y * y).T)
    tol = (131 + (K + 127) // 128) * U * size
    if c.dtype == BF:
        tol = tol + 2.0 ** -12 * root
    h = torch.finfo(c.dtype).eps / 2
    bad = ~(np.abs(f64(c) - want) <= tol * (1 + h) + h * np.abs(want))
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist())
    return want


SIZES = [(1, 16, 16), (1, 1, 128), (3, 130, 144), (16, 200, 4096), (17, 129, 1040), (32, 64, 256), (33, 48, 640), (64, 500, 2048), (65, 300, 400),
         (100, 128, 128), (128, 129, 16), (200, 1000, 1296), (257, 511, 512), (1000, 260, 272), (300, 4100, 384), (2100, 2050, 144), (4096, 3300, 208),
         (2048, 8325, 1040)]   # (the last: whole rounds of one tile and the columns left in a second launch)


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product(M, N, K, out):
    say(f"product {M} x {N} x {K} {out}")
    a, sa, w, sw = make(M, N, K, M + N + K, pad=16 if M % 2 else 0)
    guard = torch.full((M * N + 256,), 7.0, dtype=out, device="cuda")
    c = kda.gemm_fp8(a, sa, w, sw, out=guard[:M * N].view(M, N))
    again = kda.gemm_fp8(a, sa, w, sw, out_dtype=out)
    torch.cuda.synchronize()
    check(a, sa, w, sw, c)
    assert torch.equal(c, again) and bool((guard[M * N:] == 7.0).all())


def test_exact_sums():
    # small whole numbers and scales of one: every sum is exact in fp32 and in the matrix instruction
    r = np.random.default_rng(3)
    for M, N, K in ((5, 70, 272), (150, 200, 1024), (2300, 2100, 256)):
        a, w = (cast(r.integers(-3, 4, s).astype(np.float64), F32) for s in ((M, K), (N, K)))
        one = lambda *s: torch.ones(s, device="cuda")
        kb = (K + 127) // 128
        c = kda.gemm_fp8(a.to(F8).cuda(), one(M, kb), w.to(F8).cuda(), one((N + 127) // 128, kb), out_dtype=F32)
        assert torch.equal(c.cpu().double(), a.double() @ w.double().T)


def test_batch_of_tokens_and_one_row_at_a_time():
    # a row's result does not depend on how many rows run with it, within a variant's sums
    a, sa, w, sw = make(24, 300, 1280, 11)
    c = kda.gemm_fp8(a.view(2, 12, 1280), sa.view(2, 12, 10), w, sw)
    assert c.shape == (2, 12, 300)
    check(a, sa, w, sw, c.view(24, 300))
    for m in (0, 13):
        check(a[m:m + 1], sa[m:m + 1], w, sw, kda.gemm_fp8(a[m:m + 1], sa[m:m + 1], w, sw, out_dtype=F32))


@pytest.mark.parametrize("M", [4, 50, 200, 2100])
@pytest.mark.parametrize("K", [256, 272])
def test_values_that_are_not_finite_stay_in_their_row_or_column(M, K):
    N = 2100 if M == 2100 else 150
    a, sa, w, sw = make(M, N, K, 12)
    clean = kda.gemm_fp8(a, sa, w, sw)
    a, sa, w = a.clone(), sa.clone(), w.clone()
    a[1, 5] = float("nan")
    sa[2, 1] = float("inf")
    w[7, K - 1] = float("nan")
    w[9, 3] = float("nan")
    c = kda.gemm_fp8(a, sa, w, sw)
    assert torch.isnan(c[1]).all() and torch.isnan(c[:, 7]).all() and torch.isnan(c[:, 9]).all() and not torch.isfinite(c[2]).any()
    rows, cols = [m for m in range(M) if m not in (1, 2)], [n for n in range(N) if n not in (7, 9)]
    assert torch.equal(c[rows][:, cols], clean[rows][:, cols])


def test_rows_far_apart():
    # rows 2^24 bytes apart: a tile of 256 rows spans 2^32 bytes
    M, N, K = 260, 140, 256
    a, sa, w, sw = make(M, N, K, 13)
    wide = torch.empty((M, 1 << 24), dtype=torch.uint8, device="cuda").view(F8)
    wide[:, -K:] = a
    big = kda.gemm_fp8(wide[:, -K:], sa, w, sw)
    assert torch.equal(big, kda.gemm_fp8(a, sa, w, sw))


def test_refusals():
    a, sa, w, sw = make(4, 64, 256, 14)
    with pytest.raises(ValueError, match="sa must be"):
        kda.gemm_fp8(a, sa[:, :1], w, sw)
    with pytest.raises(ValueError, match="sw must be"):
        kda.gemm_fp8(a, sa, w, sw[:, :1])
    with pytest.raises(TypeError, match="float8"):
        kda.gemm_fp8(a, sa, w.float(), sw)
    with pytest.raises(TypeError):
        kda.gemm_fp8(a, sa, w, sw, out_dtype=torch.float16)
    with pytest.raises(kda.KDAError):
        kda.gemm_fp8(a[:, :248], sa, w[:, :248].contiguous(), sw)


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("M,N,K", [(33, 100, 272), (70, 520, 1296), (250, 250, 400), (4000, 9, 528), (17, 7000, 144), (16, 8200, 256), (300, 900, 1040),
                                   (90, 8300, 2064), (600, 3900, 1168)])
def test_few_outputs_and_steps_shared_by_groups(M, N, K, out):
    say(f"product {M} x {N} x {K} {out}")
    a, sa, w, sw = make(M, N, K, 17)
    c = kda.gemm_fp8(a, sa, w, sw, out_dtype=out)
    again = kda.gemm_fp8(a, sa, w, sw, out_dtype=out)
    torch.cuda.synchronize()
    check(a, sa, w, sw, c)
    assert torch.equal(c, again)


@pytest.mark.parametrize("M", [70, 300, 600])
def test_values_that_are_not_finite_in_tiles(M):
    a, sa, w, sw = make(M, 5000, 400, 18)
    clean = kda.gemm_fp8(a, sa, w, sw)
    a, sa, w = a.clone(), sa.clone(), w.clone()
    a[M - 1, 399], w[4990, 130] = float("nan"), float("nan")
    sa[3, 2] = float("inf")
    c = kda.gemm_fp8(a, sa, w, sw)
    assert torch.isnan(c[M - 1]).all() and torch.isnan(c[:, 4990]).all() and not torch.isfinite(c[3]).any()
    rows, cols = [m for m in range(M) if m not in (3, M - 1)], [n for n in range(5000) if n != 4990]
    assert torch.equal(c[rows][:, cols], clean[rows][:, cols])


def test_gradient_of_the_rows_by_the_transposed_weights():
    # dx = dc w: rows of dc in 8 bits, w and its scales transposed
    M, N, K = 300, 400, 272
    _, _, w, sw = make(M, N, K, 19)
    d8, sd, _, _ = make(M, 16, N, 20)
    dx = kda.gemm_fp8(d8, sd, w.t().contiguous(), sw.t().contiguous(), out_dtype=F32)
    torch.cuda.synchronize()
    D = f64(d8) * block.spread(f64(sd), N)
    Wf = f64(w) * block.spread(block.spread(f64(sw), K), N, 0)
    want, size = D @ Wf, np.abs(D) @ np.abs(Wf)
    # (the sums' roundings as in check, and those of the scales' products here)
    assert np.all(np.abs(f64(dx) - want) <= (131 + 4 + 2) * U * size + U * np.abs(want))


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("M,N,K", [(760, 8100, 272), (1530, 4090, 144), (1500, 8190, 400), (1537, 8193, 144)])
def test_tiles_of_192_rows(M, N, K, out):
    say(f"product {M} x {N} x {K} {out}")
    a, sa, w, sw = make(M, N, K, 21)
    check(a, sa, w, sw, kda.gemm_fp8(a, sa, w, sw, out_dtype=out))
