"""Argument checks of the operators around the recurrence (short convolution,
norms of query and key heads): every bad call is refused before anything is
enqueued, so these run without a GPU."""
import ctypes

import pytest
import torch

from gated_delta_rule_96_amd import kda

# 16-byte aligned addresses far apart, never dereferenced: a check fails first
A = [(i + 1) << 36 for i in range(12)]


def call(name, order, base, **kw):
    a = dict(base)
    a.update(kw)
    return getattr(kda.lib(), name)(*[a[n] for n in order])


CONV = dict(x=A[0], ldx=64, w=A[1], bias=A[2], s0=A[3], st=A[4], y=A[5], flags=1, dtype=1, B=2, T=10, D=64, W=4, cu=None, N=0,
            stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(w=None), 1), (dict(y=None), 1),
    (dict(B=0), 2), (dict(T=0), 2), (dict(T=(1 << 30) + 1), 2), (dict(D=0), 2), (dict(ldx=63), 2), (dict(flags=2), 2),
    (dict(dtype=2), 3), (dict(x=A[0] + 1), 4), (dict(w=A[1] + 4), 4), (dict(st=A[4] + 2), 4), (dict(y=A[5] + 8), 4),
    (dict(W=1), 5), (dict(W=5), 5),
    (dict(y=A[0]), 10), (dict(y=A[0] + 64), 10), (dict(st=A[5]), 10), (dict(st=A[3] + 16), 10), (dict(y=A[3]), 10),
])
def test_conv_fwd_refuses(kw, code):
    assert call("kda_conv_fwd", CONV, CONV, **kw) == code


def test_conv_refuses_bad_sequences():
    cu = lambda *v: (ctypes.c_int * len(v))(*v)
    for c, n, b in ((cu(0, 6, 5), 2, 1), (cu(1, 10), 1, 1), (cu(0, 9), 1, 1), (cu(0, 10), 0, 1), (cu(0, 10), 1, 2)):
        assert call("kda_conv_fwd", CONV, CONV, cu=c, N=n, B=b) == 2


STEP = dict(x=A[0], ldx=64, w=A[1], bias=None, state=A[3], so=A[3], y=A[5], flags=0, dtype=0, B=2, D=64, W=3, stream=None)


@pytest.mark.parametrize("kw,code", [(dict(state=None), 1), (dict(so=None), 1), (dict(B=0), 2), (dict(dtype=9), 3), (dict(so=A[3] + 4), 4),
                                     (dict(W=9), 5), (dict(so=A[3] + 16), 10), (dict(y=A[0]), 10), (dict(so=A[0]), 10)])
def test_conv_step_refuses(kw, code):
    assert call("kda_conv_step", STEP, STEP, **kw) == code


CBWD = dict(x=A[0], ldx=64, w=A[1], bias=None, s0=A[3], dy=A[4], gt=0, dst=A[5], dx=A[6], dw=A[7], db=A[8], ds0=A[9], flags=1, dtype=1,
            B=2, T=10, D=64, W=4, cu=None, N=0, ws=A[10], wsb=1 << 30, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(dy=None), 1), (dict(dx=None), 1), (dict(dw=None), 1), (dict(T=-1), 2), (dict(gt=3), 3), (dict(dtype=0, gt=1), 3),
    (dict(dst=A[5] + 4), 4), (dict(ws=A[10] + 16), 4), (dict(W=6), 5), (dict(ws=None), 6), (dict(wsb=16), 6),
    (dict(dx=A[4]), 10), (dict(ds0=A[5]), 10), (dict(dw=A[8]), 10), (dict(dx=A[10]), 10),
])
def test_conv_bwd_refuses(kw, code):
    assert call("kda_conv_bwd", CBWD, CBWD, **kw) == code


def test_conv_workspace_bytes():
    f = kda.lib().kda_conv_bwd_workspace_bytes
    assert f(1, 100, 64, 4, 0) > 0 and f(1, 100, 64, 4, 0) % 256 == 0
    assert f(1, 100, 64, 4, 300) >= f(1, 100, 64, 4, 0)
    for bad in ((0, 1, 1, 4, 0), (1, 0, 1, 4, 0), (1, 1, 0, 4, 0), (1, 1, 1, 5, 0), (2, 1, 1, 4, 3), (1, 1, 1, 4, -1)):
        assert f(*bad) == 0


QK = dict(q=A[0], ldq=512, k=A[1], ldk=256, wq=A[2], wk=A[3], cos=A[4], sin=A[5], pos=A[6], pos0=0, n_pos=100, eps=1e-6, qo=A[7], ko=A[8],
          flags=0, dtype=1, B=2, T=10, Hq=4, Hk=2, d=128, rot=64, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(cos=None), 1), (dict(qo=None), 1), (dict(ko=None), 1),
    (dict(B=0), 2), (dict(Hq=0), 2), (dict(ldq=504), 2), (dict(ldk=128), 2), (dict(flags=4), 2), (dict(eps=-1.0), 2),
    (dict(eps=float("nan")), 2), (dict(n_pos=0), 2), (dict(pos=None, pos0=91), 2), (dict(pos=None, pos0=-1), 2), (dict(rot=-8), 2),
    (dict(dtype=5), 3), (dict(q=A[0] + 8), 4), (dict(ldq=516), 4), (dict(sin=A[5] + 4), 4), (dict(pos=A[6] + 2), 4), (dict(ko=A[8] + 8), 4),
    (dict(d=100, ldq=400, ldk=200), 5), (dict(d=520, ldq=2080, ldk=1040), 5), (dict(rot=60), 5), (dict(rot=136), 5),
    (dict(qo=A[1]), 10), (dict(qo=A[0] + 1024), 10), (dict(ko=A[7]), 10), (dict(ldq=1024, qo=A[0]), 10), (dict(qo=A[4]), 10),
])
def test_qk_refuses(kw, code):
    assert call("kda_qk_norm_rope", QK, QK, **kw) == code


QBWD = dict(q=A[0], ldq=512, k=A[1], ldk=256, wq=A[2], wk=A[3], cos=A[4], sin=A[5], pos=A[6], pos0=0, n_pos=100, eps=1e-6, dqo=A[7], dko=A[8],
            gt=0, dq=A[9], dk=A[10], dwq=A[11], dwk=A[11] + 4096, flags=0, dtype=1, B=2, T=10, Hq=4, Hk=2, d=128, rot=64, ws=A[11] + (1 << 30),
            wsb=1 << 30, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(dqo=None), 1), (dict(dk=None), 1), (dict(gt=2), 3), (dict(dtype=0, gt=1), 3), (dict(dwk=A[11] + 4), 4), (dict(d=12), 5),
    (dict(ws=None), 6), (dict(wsb=100), 6), (dict(dq=A[7]), 10), (dict(dk=A[1]), 10), (dict(dwk=A[11]), 10),
])
def test_qk_bwd_refuses(kw, code):
    assert call("kda_qk_norm_rope_bwd", QBWD, QBWD, **kw) == code


def test_status_text():
    assert "overlap" in kda.status_str(kda.KDA_ERR_OVERLAP)


def test_binding_checks_before_the_library():
    # CPU tensors and shapes that do not fit are refused by name
    x, w = torch.zeros(1, 4, 8), torch.zeros(8, 4)
    with pytest.raises(ValueError, match="GPU"):
        kda.conv_fwd(x, w)
    with pytest.raises(ValueError, match="GPU"):
        kda.qk_norm_rope(torch.zeros(1, 2, 3, 64), None)
    with pytest.raises(ValueError, match="mode"):
        kda.qk_norm_rope(torch.zeros(1, 2, 3, 64), None, mode="max")
    with pytest.raises(ValueError, match="rise"):
        kda._packed([0, 3, 2, 4], 1, 4)
    with pytest.raises(ValueError, match="B = 1"):
        kda._packed([0, 4], 2, 4)


SSM = dict(x=A[0], ldx=256, dt=A[1], lddt=4, A=A[2], B=A[3], ldb=256, C=A[4], ldc=256, D=A[5], bias=A[6], h0=A[7], ht=A[8], y=A[9], flags=1,
           dtype=1, Bn=2, T=1000, H=4, G=2, dk=128, dv=64, cu=None, N=0, ws=A[10], wsb=1 << 34, stream=None)
SSM_ORDER = list(SSM)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(dt=None), 1), (dict(A=None), 1), (dict(B=None), 1), (dict(C=None), 1), (dict(y=None), 1),
    (dict(Bn=0), 2), (dict(T=0), 2), (dict(H=0), 2), (dict(G=3), 2), (dict(G=0), 2), (dict(ldx=255), 2), (dict(lddt=3), 2), (dict(ldb=128), 2),
    (dict(flags=2), 2), (dict(dtype=4), 3), (dict(x=A[0] + 8), 4), (dict(ldx=260), 4), (dict(dt=A[1] + 1), 4), (dict(h0=A[7] + 4), 4),
    (dict(ht=A[8] + 8), 4), (dict(ws=A[10] + 128), 4), (dict(dk=96), 5), (dict(dv=32), 5), (dict(ws=None), 6), (dict(wsb=100), 6),
    (dict(y=A[0]), 10), (dict(ht=A[7] + 16), 10), (dict(ht=A[9]), 10), (dict(y=A[10]), 10),
])
def test_ssm_fwd_refuses(kw, code):
    assert call("kda_ssm_fwd_chunked", SSM_ORDER, SSM, **kw) == code


def test_ssm_refuses_bad_sequences_and_sizes():
    cu = lambda *v: (ctypes.c_int * len(v))(*v)
    for c, n, b in ((cu(0, 600, 500), 2, 1), (cu(0, 999), 1, 1), (cu(0, 1000), 0, 1), (cu(0, 1000), 1, 2)):
        assert call("kda_ssm_fwd_chunked", SSM_ORDER, SSM, cu=c, N=n, Bn=b) == 2
    f = kda.lib().kda_ssm_workspace_bytes
    assert f(1, 100, 4, 128, 128, 1) == 0                    # one part: no states between parts
    assert f(1, 100000, 4, 128, 128, 1) % 256 == 0 and f(1, 100000, 4, 128, 128, 1) > 0
    assert f(1, 100000, 4, 96, 128, 1) == 0 and f(0, 100000, 4, 128, 128, 1) == 0


SSTEP = {k: v for k, v in SSM.items() if k not in ("T", "cu", "N", "ws", "wsb")}


@pytest.mark.parametrize("kw,code", [(dict(h0=None), 1), (dict(ht=None), 1), (dict(Bn=-1), 2), (dict(G=3), 2), (dict(dtype=2), 3), (dict(ldc=260), 4),
                                     (dict(dk=32), 5), (dict(ht=A[7] + 16), 10), (dict(y=A[8]), 10)])
def test_ssm_step_refuses(kw, code):
    assert call("kda_ssm_step", list(SSTEP), SSTEP, **kw) == code


SBWD = dict(x=A[0], ldx=256, dt=A[1], lddt=4, A=A[2], B=A[3], ldb=256, C=A[4], ldc=256, D=None, bias=None, h0=None, dy=A[5], dht=None, dx=A[6],
            ddt=A[7], dA=A[8], dB=A[9], dC=A[10], dD=None, dbias=None, dh0=None, flags=1, dtype=1, Bn=2, T=1000, H=4, G=2, dk=128, dv=64, cu=None,
            N=0, ws=A[11], wsb=1 << 40, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(dy=None), 1), (dict(dx=None), 1), (dict(ddt=None), 1), (dict(dA=None), 1), (dict(dB=None), 1), (dict(dC=None), 1), (dict(G=3), 2),
    (dict(dtype=3), 3), (dict(dht=A[0] + 4), 4), (dict(ws=A[11] + 16), 4), (dict(dv=48), 5), (dict(ws=None), 6), (dict(wsb=1000), 6),
    (dict(dx=A[5]), 10), (dict(dB=A[10]), 10), (dict(dA=A[2]), 10), (dict(dx=A[11]), 10),
])
def test_ssm_bwd_refuses(kw, code):
    assert call("kda_ssm_bwd_chunked", list(SBWD), SBWD, **kw) == code


def test_ssm_bwd_workspace_bytes():
    f = kda.lib().kda_ssm_bwd_workspace_bytes
    assert f(1, 64, 2, 1, 64, 64, 1, 0) % 256 == 0 and f(1, 6400, 2, 1, 64, 64, 1, 0) >= 100 * 2 * 2 * 64 * 64 * 4
    assert f(1, 640, 2, 1, 64, 64, 1, 50) >= f(1, 640, 2, 1, 64, 64, 1, 0)
    for bad in ((0, 1, 2, 1, 64, 64, 1, 0), (1, 1, 2, 3, 64, 64, 1, 0), (1, 1, 2, 1, 32, 64, 1, 0), (1, 1, 2, 1, 64, 64, 2, 0), (2, 1, 2, 1, 64, 64, 1, 3)):
        assert f(*bad) == 0


@pytest.mark.parametrize("kw", [dict(Hq=(1 << 31) - 1, Hk=0, k=None, ko=None, d=8, rot=0), dict(Hq=1, Hk=(1 << 31) - 1, d=8, rot=0),
                                dict(Hq=(1 << 24) + 1, Hk=0, k=None, ko=None, d=8, rot=0)])
def test_qk_refuses_more_heads_than_it_numbers(kw):
    # heads are numbered in 32 bits, up to a wave's 32 beyond the last one
    one = dict(B=1, T=1, ldq=8 * kw["Hq"], ldk=8 * kw["Hk"], **kw)
    assert call("kda_qk_norm_rope", QK, QK, **one) == 2
    back = dict(one, dk=one.get("ko", QBWD["dk"]), dko=None if kw["Hk"] == 0 else QBWD["dko"])
    back.pop("ko", None)
    assert call("kda_qk_norm_rope_bwd", QBWD, QBWD, **back) == 2
    assert kda.lib().kda_qk_bwd_workspace_bytes(1, 1, kw["Hq"], kw["Hk"], 8) == 0


FAR = [(i + 1) << 45 for i in range(14)]   # addresses with room for hundreds of gigabytes


def far(base):
    """The base call with its pointers far apart."""
    return {n: FAR[A.index(v)] if v in A else v for n, v in base.items()}


def test_sizes_beyond_a_launch_are_refused():
    # a launch of 2^32 threads runs only a part of them: refused as a size,
    # before anything is enqueued
    many, none = (1 << 31) - 1, dict(h0=None, ht=None, dk=64, dv=64, H=1, G=1, ldx=64, lddt=1, ldb=64, ldc=64)
    assert call("kda_conv_fwd", CONV, far(CONV), B=many, T=1, D=3, ldx=3, s0=None, st=None) == 2
    assert call("kda_conv_step", STEP, far(STEP), B=many, D=9, ldx=9) == 2
    one = dict(B=1, T=1, D=60_000_000, ldx=60_000_000, s0=None, dst=None, ds0=None, wsb=1 << 44)
    assert call("kda_conv_bwd", CBWD, far(CBWD), **one) == 2                                         # (the sums of dw)
    assert call("kda_conv_bwd", CBWD, far(CBWD), **dict(one, B=many, D=7, ldx=7)) == 2
    assert call("kda_ssm_fwd_chunked", SSM_ORDER, far(SSM), Bn=1 << 23, T=1, **none) == 2
    assert call("kda_ssm_step", list(SSTEP), far(SSTEP), Bn=1 << 23, **dict(none, h0=FAR[12], ht=FAR[12])) == 2
    back = {n: v for n, v in none.items() if n != "ht"}
    assert call("kda_ssm_bwd_chunked", list(SBWD), far(SBWD), Bn=1 << 23, T=1, wsb=1 << 44, **back) == 2
    cu = (ctypes.c_int * 301)(*[0] * 300, 1000)
    wide = dict(none, H=1 << 18, ldx=1 << 24, lddt=1 << 18)   # 128 sequences a launch of too many heads
    assert call("kda_ssm_fwd_chunked", SSM_ORDER, far(SSM), Bn=1, T=1000, cu=cu, N=300, **wide, wsb=1 << 44) == 2


def test_binding_refuses_what_32_bits_do_not_hold():
    # sizes and positions go to the library as 32-bit ints: none may wrap around
    with pytest.raises(ValueError, match="32 bits"):
        kda._packed([0, (1 << 32) + 4], 1, 4)
    with pytest.raises(ValueError, match="32 bits"):
        kda.varlen_snapshots([0, (1 << 32) + 640], 1)
    x = torch.empty((1, (1 << 32) + 3, 8), dtype=torch.bfloat16, device="meta")
    with pytest.raises(ValueError, match="32 bits"):
        kda._rows(x, "x", (1, (1 << 32) + 3), (8,))
    q = torch.empty((1, 4, 1, 64), device="meta")
    for kw in (dict(pos0=1 << 32), dict(pos0=-(1 << 31) - 1)):
        with pytest.raises(ValueError, match="32 bits"):
            kda.qk_norm_rope(q, None, cos=torch.empty((8, 8)), sin=torch.empty((8, 8)), **kw)
    long = torch.empty(((1 << 32) + 8, 8), device="meta")
    with pytest.raises(ValueError, match="32 bits"):
        kda.qk_norm_rope(q, None, cos=long, sin=long)


def test_workspace_sizes_of_absurd_calls_are_zero():
    # sizes the calls refuse: 0, not a byte count that wrapped around
    many = (1 << 31) - 1
    L = kda.lib()
    assert L.kda_ssm_bwd_workspace_bytes(1, 64, 1 << 18, 1, 128, 128, 1, many) == 0
    assert L.kda_conv_bwd_workspace_bytes(1, 1, many, 4, many) == 0 and L.kda_conv_bwd_workspace_bytes(1, 1, many, 4, 0) == 0


def test_stream_without_the_raw_handle(monkeypatch):
    # a torch without the private accessor: the public stream's handle
    class Stream:
        cuda_stream = 1234
    asked = []
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: asked.append(d) or Stream())
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    assert kda._stream(torch.device("cuda", 3)) == 1234 and asked == [torch.device("cuda", 3)]
