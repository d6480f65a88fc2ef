"""Python binding of libkda.so: marshals torch device tensors into the C ABI
declared in include/kda.h.  Every step of the computation runs in the HIP
kernels; this module only checks tensor metadata, allocates outputs with
torch (device memory plumbing) and passes pointers plus the current stream.

Raises KDAError (with the library's status string) on any non-zero status,
and RuntimeError if the library has not been built.
"""
from __future__ import annotations

import ctypes
import math
from pathlib import Path

import torch

PKG = Path(__file__).resolve().parent
LIB_PATH = PKG / "libkda.so"
# profiling build with the fused prefill's cycle stamps (include/kda_stamps.h);
# set LIB_PATH to it before the first call to use it
STAMPS_LIB_PATH = PKG / "libkda_stamps.so"
STAMP_WGS, STAMP_WAVES, STAMP_SLOTS, STAMP_ROLE, STAMP_COUNT = 256, 8, 32, 29, 30

KDA_F32, KDA_BF16 = 0, 1
KDA_ERR_UNSUPPORTED, KDA_ERR_RANGE, KDA_ERR_INCOMPLETE, KDA_ERR_OVERLAP = 5, 7, 9, 10
KDA_STAGES_UNBOUNDED = 4
KDA_LAYER_QK_L2NORM = 1
KDA_CONV_SILU = 1
KDA_QK_RMS, KDA_QK_INTERLEAVED = 1, 2
KDA_SSM_SOFTPLUS = 1
KDA_LRU_UNIT = 1
CHUNK = 64
GMIN = -5.0

_lib = None


class KDAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: status {status} ({status_str(status)})")


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        if not LIB_PATH.exists():
            raise RuntimeError(f"{LIB_PATH} is missing: run __graft_entry__.build() "
                               "(python -m gated_delta_rule_96_amd.build) first")
        L = ctypes.CDLL(str(LIB_PATH))
        P, I, F, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        L.kda_abi_version.restype = I
        L.kda_abi_version.argtypes = []
        L.kda_status_str.restype = ctypes.c_char_p
        L.kda_status_str.argtypes = [I]
        L.kda_prepare_decay.restype = I
        L.kda_prepare_decay.argtypes = [P, P, F, P, P, I, I, I, I, I, I, P]
        L.kda_prepare_decay_softplus.restype = I
        L.kda_prepare_decay_softplus.argtypes = [P, P, P, P, I, I, I, I, I, I, P]
        L.kda_fwd_workspace_bytes.restype = S
        L.kda_fwd_workspace_bytes.argtypes = [I, I, I, I, I, I, I]
        L.kda_fwd_stages_workspace_bytes.restype = S
        L.kda_fwd_stages_workspace_bytes.argtypes = [I, I, I, I, I, I, I]
        L.kda_fwd_chunked.restype = I
        L.kda_fwd_chunked.argtypes = [P, P, P, P, P, P, F, P, P, P, I, I, I, I, I, I, I, P, S, P]
        L.kda_fwd_chunked_layer.restype = I
        L.kda_fwd_chunked_layer.argtypes = [P, P, P, P, P, P, P, F, P, P, P, I, I, I, I, I, I, I, I, P, S, P]
        L.kda_fwd_chunked_varlen.restype = I
        L.kda_fwd_chunked_varlen.argtypes = [P, P, P, P, P, P, F, P, I, P, P, P, P, I, I, I, I, I, I, I, P, S, P]
        L.kda_fwd_varlen_snapshots.restype = ctypes.c_longlong
        L.kda_fwd_varlen_snapshots.argtypes = [P, I, I, I]
        L.kda_fwd_chunked_noalloc.restype = I
        L.kda_fwd_chunked_noalloc.argtypes = [P, P, P, P, P, P, F, P, P, P, I, I, I, I, I, I, I, P]
        L.kda_fwd_chunked_unbounded.restype = I
        L.kda_fwd_chunked_unbounded.argtypes = [P, P, P, P, P, P, F, P, P, P, I, I, I, I, I, I, I, P, S, P]
        L.kda_fwd_chunked_stages.restype = I
        L.kda_fwd_chunked_stages.argtypes = [P, P, P, P, P, P, F, P, P, P, I, I, I, I, I, I, I, P, S, I, P]
        L.kda_decode_step.restype = I
        L.kda_decode_step.argtypes = [P, P, P, P, P, F, P, P, I, I, I, I, I, P]
        L.kda_decode_step_layer.restype = I
        L.kda_decode_step_layer.argtypes = [P, P, P, P, P, P, P, F, P, P, I, I, I, I, I, I, P]
        L.kda_bwd_workspace_bytes.restype = S
        L.kda_bwd_workspace_bytes.argtypes = [I, I, I, I, I, I, I]
        L.kda_bwd_chunked.argtypes = [P, P, P, P, P, F, P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, P, S, P]
        L.kda_fwd_status.restype = I
        L.kda_fwd_status.argtypes = [P, P]
        L.kda_fwd_status_word.restype = P
        L.kda_fwd_status_word.argtypes = [P]
        LL = ctypes.c_longlong
        for name, res, args in (
                ("kda_conv_fwd", I, [P, LL, P, P, P, P, P, I, I, I, I, I, I, P, I, P]),
                ("kda_conv_step", I, [P, LL, P, P, P, P, P, I, I, I, I, I, P]),
                ("kda_conv_bwd_workspace_bytes", S, [I, I, I, I, I]),
                ("kda_conv_bwd", I, [P, LL, P, P, P, P, I, P, P, P, P, P, I, I, I, I, I, I, P, I, P, S, P]),
                ("kda_qk_norm_rope", I, [P, LL, P, LL, P, P, P, P, P, I, I, F, P, P] + [I] * 8 + [P]),
                ("kda_qk_bwd_workspace_bytes", S, [I, I, I, I, I]),
                ("kda_qk_norm_rope_bwd", I, [P, LL, P, LL, P, P, P, P, P, I, I, F, P, P, I, P, P, P, P] + [I] * 8 + [P, S, P]),
                ("kda_ssm_workspace_bytes", S, [I] * 6),
                ("kda_ssm_fwd_chunked", I, [P, LL, P, LL, P, P, LL, P, LL, P, P, P, P, P] + [I] * 8 + [P, I, P, S, P]),
                ("kda_ssm_step", I, [P, LL, P, LL, P, P, LL, P, LL, P, P, P, P, P] + [I] * 7 + [P]),
                ("kda_ssm_bwd_workspace_bytes", S, [I] * 8),
                ("kda_add_rms_norm", I, [P, LL, P, LL, I, P, F, P, P, P, I, LL, I, P]),
                ("kda_add_rms_norm_bwd_workspace_bytes", S, [LL, I]),
                ("kda_add_rms_norm_bwd", I, [P, LL, P, F, P, I, P, P, P, I, LL, I, P, S, P]),
                ("kda_gemm_fp8", I, [P, LL, P, LL, P, P, P, I, LL, I, I, P]),
                ("kda_lru_workspace_bytes", S, [I] * 4),
                ("kda_lru_fwd", I, [P, LL, P, LL, P, LL, P, P, P, P, I, I, I, I, I, P, I, P, S, P]),
                ("kda_lru_step", I, [P, LL, P, LL, P, LL, P, P, P, P, I, I, I, I, P]),
                ("kda_lru_bwd_workspace_bytes", S, [I] * 4),
                ("kda_lru_bwd", I, [P, LL, P, LL, P, LL] + [P] * 9 + [I] * 5 + [P, I, P, S, P]),
                ("kda_ssm_bwd_chunked", I, [P, LL, P, LL, P, P, LL, P, LL] + [P] * 13 + [I] * 8 + [P, I, P, S, P])):
            getattr(L, name).restype = res
            getattr(L, name).argtypes = args
        if hasattr(L, "kda_stamps_read"):
            L.kda_stamps_read.restype = I
            L.kda_stamps_read.argtypes = [P, S]
        _lib = L
    return _lib


def status_str(s: int) -> str:
    return lib().kda_status_str(int(s)).decode()


def abi_version() -> int:
    return lib().kda_abi_version()


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return KDA_BF16
    if t.dtype == torch.float32:
        return KDA_F32
    raise TypeError(f"unsupported dtype {t.dtype} (bfloat16 or float32)")


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must live on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(device) -> int:
    # (the handle itself where torch gives it: torch.cuda.current_stream()
    # builds an object around it, 1.9 us of a single-token call's 12)
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return torch.cuda.current_stream(device).cuda_stream if raw is None else raw(device.index)


def _check(status: int, where: str):
    if status != 0:
        raise KDAError(status, where)


def prepare_decay(z=None, A=None, g=None, *, want_g=True, want_gcum=True, gmin=GMIN, chunk=CHUNK,
                  softplus=False):
    """Gate mode: prepare_decay(z, A) -> (g, gcum); scan mode: prepare_decay(g=g) -> gcum.
    z, g: [B, T, H, dk] (bf16 or fp32); A: [H] fp32.  softplus=True: the
    unbounded gate g = -Softplus(exp(A) z) (kda_prepare_decay_softplus)."""
    if z is not None:
        B, T, H, dk = z.shape
        dt = _dtype_code(z)
        if A is None or A.dtype != torch.float32 or A.shape != (H,):
            raise ValueError("A must be fp32 [H]")
        g_out = torch.empty_like(z) if want_g else None
        gcum = torch.empty(z.shape, dtype=torch.float32, device=z.device) if want_gcum else None
        if softplus:
            _check(lib().kda_prepare_decay_softplus(_ptr(z), _ptr(A), _ptr(g_out), _ptr(gcum), dt, B, T, H, dk,
                                                    chunk, _stream(z.device)), "kda_prepare_decay_softplus")
        else:
            _check(lib().kda_prepare_decay(_ptr(z), _ptr(A), gmin, _ptr(g_out), _ptr(gcum), dt, B, T, H, dk,
                                           chunk, _stream(z.device)), "kda_prepare_decay")
        return g_out, gcum
    if g is None:
        raise ValueError("need z (gate mode) or g (scan mode)")
    B, T, H, dk = g.shape
    gcum = torch.empty(g.shape, dtype=torch.float32, device=g.device)
    _check(lib().kda_prepare_decay(None, None, gmin, _ptr(g), _ptr(gcum), _dtype_code(g), B, T, H, dk, chunk,
                                   _stream(g.device)), "kda_prepare_decay")
    return gcum


def fwd_workspace_bytes(B, T, H, dk, dv, dtype=torch.bfloat16, chunk=CHUNK, stages=False) -> int:
    """Workspace bytes of kda_fwd_chunked (stages=False) or kda_fwd_chunked_stages."""
    code = KDA_BF16 if dtype == torch.bfloat16 else KDA_F32
    f = lib().kda_fwd_stages_workspace_bytes if stages else lib().kda_fwd_workspace_bytes
    return int(f(B, T, H, dk, dv, chunk, code))


def alloc_workspace(B, T, H, dk, dv, dtype=torch.bfloat16, device="cuda", chunk=CHUNK, stages=False) -> torch.Tensor:
    n = fwd_workspace_bytes(B, T, H, dk, dv, dtype, chunk, stages)
    if n == 0:
        raise ValueError("unsupported sizes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def workspace_error(workspace: torch.Tensor) -> int:
    """Status of the last call on a workspace of a prefill, of its backward or
    of lru_fwd through kda_fwd_status: 0, or KDA_ERR_INCOMPLETE (9) when a
    hand-off wait expired and the outputs are incomplete.  Synchronises the
    current stream."""
    s = int(lib().kda_fwd_status(_ptr(workspace), _stream(workspace.device)))
    if s not in (0, KDA_ERR_INCOMPLETE):
        raise KDAError(s, "kda_fwd_status")
    return s


def check_workspace(workspace: torch.Tensor, where: str = "kda_fwd_status"):
    """Raises KDAError(KDA_ERR_INCOMPLETE) if the last call on `workspace`
    did not complete (synchronises the current stream)."""
    _check(workspace_error(workspace), where)


def fwd_chunked(q, k, v, g, beta, h0=None, *, gcum=None, scale=None, final_state=True, ht=None,
                workspace=None, out=None, chunk=CHUNK, stages=None, unbounded=False, check=False):
    """o, ht = fwd_chunked(q, k, v, g, beta, h0).  q,k,g [B,T,H,dk]; v [B,T,H,dv];
    beta [B,T,H] (bf16 or fp32); h0/ht [B,H,dk,dv] fp32; o [B,T,H,dv] fp32.
    ht may be h0 itself (in-place carry).  stages=None runs the fused
    single-pass schedule (kda_fwd_chunked); stages in {1, 2, 3} runs the
    two-kernel schedule (kda_fwd_chunked_stages) with that stage mask.
    unbounded=True: the log-decay has no lower bound (kda_fwd_chunked_unbounded,
    or KDA_STAGES_UNBOUNDED added to the stage mask).  check=True synchronises
    and raises KDAError if the fused call did not complete (kda_fwd_status)."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    for name, t in (("k", k), ("v", v), ("beta", beta)) + ((("g", g),) if g is not None else ()):
        if t.dtype != q.dtype:
            raise TypeError(f"{name} dtype {t.dtype} != q dtype {q.dtype}")
    if scale is None:
        scale = 1.0 / math.sqrt(dk)
    if workspace is None:
        workspace = alloc_workspace(B, T, H, dk, dv, q.dtype, q.device, chunk, stages is not None)
    o = torch.empty((B, T, H, dv), dtype=torch.float32, device=q.device) if out is None else out
    if o.dtype != torch.float32 or o.shape != (B, T, H, dv):
        raise ValueError("out must be fp32 [B, T, H, dv]")
    if final_state and ht is None:
        ht = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    for t in (h0, ht):
        if t is not None and (t.dtype != torch.float32 or t.shape != (B, H, dk, dv)):
            raise ValueError("states must be fp32 [B, H, dk, dv]")
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(gcum), _ptr(beta), float(scale), _ptr(h0),
            _ptr(ht if final_state else None), _ptr(o), dt, B, T, H, dk, dv, chunk, _ptr(workspace),
            workspace.numel())
    if stages is None:
        fn = lib().kda_fwd_chunked_unbounded if unbounded else lib().kda_fwd_chunked
        _check(fn(*args, _stream(q.device)), "kda_fwd_chunked_unbounded" if unbounded else "kda_fwd_chunked")
        if check:
            check_workspace(workspace, "kda_fwd_chunked")
    else:
        mask = int(stages) | (KDA_STAGES_UNBOUNDED if unbounded else 0)
        _check(lib().kda_fwd_chunked_stages(*args, mask, _stream(q.device)), "kda_fwd_chunked_stages")
    return o, (ht if final_state else None)


def fwd_chunked_layer(q, k, v, z, A, beta, h0=None, *, og=None, qk_l2norm=False, scale=None, final_state=True,
                      ht=None, workspace=None, out=None, chunk=CHUNK, check=False):
    """o, ht = fwd_chunked_layer(q, k, v, z, A, beta, h0): kda_fwd_chunked with
    the decay gate of z (A [H] fp32) fused into the kernel's scan, optional
    in-kernel q/k row L2 normalisation and optional sigmoid output gate og
    [B,T,H,dv] (same dtype as q)."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    for name, t in (("k", k), ("v", v), ("z", z), ("beta", beta)) + ((("og", og),) if og is not None else ()):
        if t.dtype != q.dtype:
            raise TypeError(f"{name} dtype {t.dtype} != q dtype {q.dtype}")
    if A.dtype != torch.float32 or A.shape != (H,):
        raise ValueError("A must be fp32 [H]")
    if scale is None:
        scale = 1.0 / math.sqrt(dk)
    if workspace is None:
        workspace = alloc_workspace(B, T, H, dk, dv, q.dtype, q.device, chunk)
    o = torch.empty((B, T, H, dv), dtype=torch.float32, device=q.device) if out is None else out
    if final_state and ht is None:
        ht = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    flags = KDA_LAYER_QK_L2NORM if qk_l2norm else 0
    _check(lib().kda_fwd_chunked_layer(_ptr(q), _ptr(k), _ptr(v), _ptr(z), _ptr(A), _ptr(beta), _ptr(og),
                                       float(scale), _ptr(h0), _ptr(ht if final_state else None), _ptr(o), flags,
                                       dt, B, T, H, dk, dv, chunk, _ptr(workspace), workspace.numel(),
                                       _stream(q.device)), "kda_fwd_chunked_layer")
    if check:
        check_workspace(workspace, "kda_fwd_chunked_layer")
    return o, (ht if final_state else None)


_INT_MAX = (1 << 31) - 1   # sizes go to the library as C ints, which ctypes would wrap around


def _cu_array(cu_seqlens):
    cu = [int(x) for x in cu_seqlens]
    if cu and (max(cu) > _INT_MAX or min(cu) < -_INT_MAX):
        raise ValueError("cu_seqlens must be in 32 bits")
    return (ctypes.c_int * len(cu))(*cu), len(cu) - 1


def varlen_snapshots(cu_seqlens, snap_every, chunk=CHUNK) -> int:
    """Number of snapshots fwd_chunked_varlen writes (kda_fwd_varlen_snapshots)."""
    arr, n = _cu_array(cu_seqlens)
    s = int(lib().kda_fwd_varlen_snapshots(ctypes.cast(arr, ctypes.c_void_p), n, int(snap_every), chunk))
    if s < 0:
        raise ValueError("invalid cu_seqlens or snap_every")
    return s


def fwd_chunked_varlen(q, k, v, g, beta, cu_seqlens, h0=None, *, gcum=None, scale=None, snap_every=0, ht=None,
                       workspace=None, out=None, chunk=CHUNK, check=False):
    """o, ht, snaps = fwd_chunked_varlen(q, k, v, g, beta, cu_seqlens, h0).
    N sequences packed along tokens: q,k,g [1,T,H,dk]; v [1,T,H,dv]; beta
    [1,T,H]; cu_seqlens host ints (N+1, from 0 to T); h0/ht [N,H,dk,dv] fp32.
    snaps [S,H,dk,dv] fp32: the state after every snap_every chunks of each
    sequence (before its end), sequences in order (None when snap_every=0)."""
    _, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    arr, N = _cu_array(cu_seqlens)
    if scale is None:
        scale = 1.0 / math.sqrt(dk)
    if workspace is None:
        workspace = alloc_workspace(1, T, H, dk, dv, q.dtype, q.device, chunk)
    o = torch.empty((1, T, H, dv), dtype=torch.float32, device=q.device) if out is None else out
    if ht is None:
        ht = torch.empty((N, H, dk, dv), dtype=torch.float32, device=q.device)
    for t in (h0, ht):
        if t is not None and (t.dtype != torch.float32 or t.shape != (N, H, dk, dv)):
            raise ValueError("states must be fp32 [N, H, dk, dv]")
    snaps = None
    if snap_every > 0:
        ns = varlen_snapshots(cu_seqlens, snap_every, chunk)
        snaps = torch.empty((max(ns, 1), H, dk, dv), dtype=torch.float32, device=q.device)
    _check(lib().kda_fwd_chunked_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(gcum), _ptr(beta), float(scale),
                                        ctypes.cast(arr, ctypes.c_void_p), N, _ptr(h0), _ptr(ht), _ptr(o),
                                        _ptr(snaps), int(snap_every), dt, T, H, dk, dv, chunk, _ptr(workspace),
                                        workspace.numel(), _stream(q.device)), "kda_fwd_chunked_varlen")
    if check:
        check_workspace(workspace, "kda_fwd_chunked_varlen")
    if snaps is not None:
        snaps = snaps[:varlen_snapshots(cu_seqlens, snap_every, chunk)]
    return o, ht, snaps


def bwd_workspace_bytes(B, T, H, dk, dv, dtype=torch.bfloat16, chunk=CHUNK) -> int:
    dt = _dtype_code(torch.empty(0, dtype=dtype))
    n = int(lib().kda_bwd_workspace_bytes(B, T, H, dk, dv, chunk, dt))
    if n == 0:
        raise KDAError(5, "kda_bwd_workspace_bytes")
    return n


def bwd_chunked(q, k, v, g, beta, h0, do, dht=None, *, scale=None, want_dh0=True, workspace=None, out=None,
                chunk=CHUNK, check=False):
    """Gradients of kda_fwd_chunked (kda_bwd_chunked): q, k, g [B,T,H,dk] and
    v [B,T,H,dv], beta [B,T,H] (bf16 or fp32), h0 [B,H,dk,dv] fp32 or None;
    do = dL/do [B,T,H,dv] fp32, dht = dL/dht [B,H,dk,dv] fp32 or None.
    Returns a dict of fp32 tensors dq, dk, dv, dg, dbeta and dh0 (None unless
    want_dh0).  `out` may supply that dict to be filled in place.  check=True
    synchronises and raises KDAError if the forward recompute did not
    complete."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    for name, t in (("k", k), ("v", v), ("g", g), ("beta", beta)):
        if t.dtype != q.dtype:
            raise TypeError(f"{name} dtype {t.dtype} != q dtype {q.dtype}")
    for name, t, shape in (("do", do, (B, T, H, dv)), ("dht", dht, (B, H, dk, dv)), ("h0", h0, (B, H, dk, dv))):
        if t is not None and (t.dtype != torch.float32 or tuple(t.shape) != shape):
            raise ValueError(f"{name} must be fp32 {list(shape)}")
    if scale is None:
        scale = 1.0 / math.sqrt(dk)
    if workspace is None:
        n = bwd_workspace_bytes(B, T, H, dk, dv, q.dtype, chunk)
        workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
    dev = q.device
    if out is None:
        out = {"dq": torch.empty((B, T, H, dk), dtype=torch.float32, device=dev),
               "dk": torch.empty((B, T, H, dk), dtype=torch.float32, device=dev),
               "dv": torch.empty((B, T, H, dv), dtype=torch.float32, device=dev),
               "dg": torch.empty((B, T, H, dk), dtype=torch.float32, device=dev),
               "dbeta": torch.empty((B, T, H), dtype=torch.float32, device=dev),
               "dh0": torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev) if want_dh0 else None}
    _check(lib().kda_bwd_chunked(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), float(scale), _ptr(h0), _ptr(do),
                                 _ptr(dht), _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["dg"]),
                                 _ptr(out["dbeta"]), _ptr(out.get("dh0")), dt, B, T, H, dk, dv, chunk,
                                 _ptr(workspace), workspace.numel(), _stream(dev)), "kda_bwd_chunked")
    if check:
        check_workspace(workspace, "kda_bwd_chunked (forward recompute)")
    return out


def decode_step(q, k, v, g, beta, state, *, scale=None, out=None):
    """o = decode_step(q, k, v, g, beta, state); state [B,H,dk,dv] fp32 is updated in place.
    q,k,g [B,H,dk]; v [B,H,dv]; beta [B,H]; o [B,H,dv] fp32."""
    B, H, dk = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    if scale is None:
        scale = 1.0 / math.sqrt(dk)
    if state.dtype != torch.float32 or state.shape != (B, H, dk, dv):
        raise ValueError("state must be fp32 [B, H, dk, dv]")
    o = torch.empty((B, H, dv), dtype=torch.float32, device=q.device) if out is None else out
    if o.dtype != torch.float32 or o.shape != (B, H, dv):
        raise ValueError("out must be fp32 [B, H, dv]")
    _check(lib().kda_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), float(scale), _ptr(state),
                                 _ptr(o), dt, B, H, dk, dv, _stream(q.device)), "kda_decode_step")
    return o


def decode_step_layer(q, k, v, z, A, beta, state, *, og=None, qk_l2norm=False, scale=None, out=None):
    """o = decode_step_layer(q, k, v, z, A, beta, state): decode_step with the
    decay gate of z (A [H] fp32), optional q/k row L2 normalisation and an
    optional sigmoid output gate og [B,H,dv] (same dtype as q) fused in;
    state [B,H,dk,dv] fp32 is updated in place."""
    B, H, dk = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    for name, t in (("k", k), ("v", v), ("z", z), ("beta", beta)) + ((("og", og),) if og is not None else ()):
        if t.dtype != q.dtype:
            raise TypeError(f"{name} dtype {t.dtype} != q dtype {q.dtype}")
    if A.dtype != torch.float32 or A.shape != (H,):
        raise ValueError("A must be fp32 [H]")
    if og is not None and og.shape != (B, H, dv):
        raise ValueError("og must be [B, H, dv]")
    if scale is None:
        scale = 1.0 / math.sqrt(dk)
    if state.dtype != torch.float32 or state.shape != (B, H, dk, dv):
        raise ValueError("state must be fp32 [B, H, dk, dv]")
    o = torch.empty((B, H, dv), dtype=torch.float32, device=q.device) if out is None else out
    if o.dtype != torch.float32 or o.shape != (B, H, dv):
        raise ValueError("out must be fp32 [B, H, dv]")
    flags = KDA_LAYER_QK_L2NORM if qk_l2norm else 0
    _check(lib().kda_decode_step_layer(_ptr(q), _ptr(k), _ptr(v), _ptr(z), _ptr(A), _ptr(beta), _ptr(og),
                                       float(scale), _ptr(state), _ptr(o), flags, dt, B, H, dk, dv,
                                       _stream(q.device)), "kda_decode_step_layer")
    return o


# ---------------------------------------------------------------- operators around the recurrence
def _rows(t, name, lead, inner):
    """Pointer and token stride of an input [*lead, *inner] that may be a slice
    of a wider tensor: inner elements contiguous, all tokens one distance apart."""
    if t.shape != lead + inner:
        raise ValueError(f"{name} must be {list(lead + inner)}, got {list(t.shape)}")
    if t.numel() > _INT_MAX and max(t.shape) > _INT_MAX:
        raise ValueError(f"{name}: a size is not in 32 bits: {list(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on the GPU")
    if t.is_contiguous():
        return t.data_ptr(), math.prod(inner)
    st, n = t.stride(), 1
    for size, stride in zip(reversed(inner), reversed(st[len(lead):])):
        if size != 1 and stride != n:
            raise ValueError(f"{name}: the elements of a token must be contiguous")
        n *= size
    ld = n
    if len(lead) == 1:
        ld = st[0] if lead[0] > 1 else n
    elif lead[1] > 1:
        ld = st[1]
        if lead[0] > 1 and st[0] != lead[1] * ld:
            raise ValueError(f"{name}: tokens must be one distance apart across the batch")
    elif lead[0] > 1:
        ld = st[0]
    if ld < n:
        raise ValueError(f"{name}: tokens overlap (an expanded tensor?)")
    return t.data_ptr(), ld


def _dense(t, name, shape, dtype, dev=None):
    """Pointer of a contiguous tensor of this shape and type, and on device dev
    if given (None passes)."""
    if t is None:
        return None
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} is on {t.device}, not on {dev}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.is_contiguous() and t.is_cuda:
        return t.data_ptr()
    return _ptr(t)   # (says which)


def _same_device(dev, **tensors):
    for n, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{n} is on {t.device}, not on {dev}")


def _call(dev, name, *args):
    """Calls entry point `name` on dev's current stream (with dev the current device)."""
    index = dev.index
    if index is None or index == _current_device():
        status = getattr(_lib or lib(), name)(*args, _stream(dev))
        if status:
            _check(status, name)
    else:
        with torch.cuda.device(dev):
            _check(getattr(lib(), name)(*args, _stream(dev)), name)


def _packed(cu_seqlens, B, T):
    """(host array or None, sequences) of a call's cu_seqlens."""
    if cu_seqlens is None:
        return None, B
    arr, n = _cu_array(cu_seqlens)
    if B != 1:
        raise ValueError("packed sequences need B = 1")
    if n < 1 or arr[0] != 0 or arr[n] != T or any(arr[i + 1] < arr[i] for i in range(n)):
        raise ValueError(f"cu_seqlens must rise from 0 to {T}")
    return arr, n


def _given(out, like, name):
    """`out` checked, or a new tensor of like's shape, type and device."""
    if out is None:
        return torch.empty_like(like, memory_format=torch.contiguous_format)
    _dense(out, name, like.shape, like.dtype, like.device)
    return out


def _scratch(workspace, nbytes, dev, name):
    if workspace is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=dev)
    if workspace.dtype != torch.uint8 or workspace.numel() < nbytes:
        raise ValueError(f"workspace must be uint8 of at least {name} = {nbytes} bytes")
    return workspace


def conv_fwd(x, w, bias=None, s0=None, *, silu=True, cu_seqlens=None, final_state=True, st=None, out=None):
    """y, st = conv_fwd(x, w, bias, s0): short causal depthwise convolution
    (kda_conv_fwd).  x [B,T,D] (bf16 or fp32, may be a slice of a wider
    tensor); w [D,W] and bias [D] fp32, W in 2..4; s0 / st [N,W-1,D] of x's
    type, the tokens before / the last tokens of each of the N = B sequences,
    or of those cu_seqlens (host ints) cuts the packed axis into; st may be s0
    itself.  silu: y = z Sigmoid(z)."""
    B, T, D = x.shape
    W = w.shape[-1]
    dt = _dtype_code(x)
    px, ld = _rows(x, "x", (B, T), (D,))
    arr, N = _packed(cu_seqlens, B, T)
    _same_device(x.device, w=w, bias=bias, s0=s0, st=st, out=out)
    y = _given(out, x, "out")
    if final_state and st is None:
        st = torch.empty((N, W - 1, D), dtype=x.dtype, device=x.device)
    _call(x.device, "kda_conv_fwd", px, ld, _dense(w, "w", (D, W), torch.float32), _dense(bias, "bias", (D,), torch.float32),
          _dense(s0, "s0", (N, W - 1, D), x.dtype), _dense(st if final_state else None, "st", (N, W - 1, D), x.dtype),
          y.data_ptr(), KDA_CONV_SILU if silu else 0, dt, B, T, D, W, arr, N)
    return y, (st if final_state else None)


def conv_step(x, w, bias, state, *, silu=True, state_out=None, out=None):
    """y = conv_step(x, w, bias, state): one token x [B,D] per sequence
    against its state [B,W-1,D], which moves on in place, or into state_out
    (the old state is then kept)."""
    B, D = x.shape
    W = w.shape[-1]
    px, ld = _rows(x, "x", (B,), (D,))
    dev, st = x.device, (B, W - 1, D)
    y = _given(out, x, "out")
    so = state if state_out is None else state_out
    _call(dev, "kda_conv_step", px, ld, _dense(w, "w", (D, W), torch.float32, dev), _dense(bias, "bias", (D,), torch.float32, dev),
          _dense(state, "state", st, x.dtype, dev), _dense(so, "state_out", st, x.dtype, dev), y.data_ptr(),
          KDA_CONV_SILU if silu else 0, _dtype_code(x), B, D, W)
    return y


def conv_bwd(x, w, bias, dy, s0=None, dst=None, *, silu=True, cu_seqlens=None, workspace=None, out=None):
    """Gradients of conv_fwd (kda_conv_bwd) from dy [B,T,D] (x's type or fp32)
    and dst [N,W-1,D] (gradient of st, or None): a dict of dx (x's type), dw
    [D,W] and dbias [D] fp32 (None without a bias) and ds0 [N,W-1,D] (None
    without s0).  `out` may supply that dict to be filled in place."""
    B, T, D = x.shape
    W = w.shape[-1]
    dev = x.device
    px, ld = _rows(x, "x", (B, T), (D,))
    arr, N = _packed(cu_seqlens, B, T)
    dt, gt = _dtype_code(x), _dtype_code(dy)
    if out is None:
        out = {"dx": torch.empty((B, T, D), dtype=x.dtype, device=dev), "dw": torch.empty((D, W), dtype=torch.float32, device=dev),
               "dbias": torch.empty(D, dtype=torch.float32, device=dev) if bias is not None else None,
               "ds0": torch.empty((N, W - 1, D), dtype=x.dtype, device=dev) if s0 is not None else None}
    ws = _scratch(workspace, lib().kda_conv_bwd_workspace_bytes(B, T, D, W, N if arr is not None else 0), dev,
                  "kda_conv_bwd_workspace_bytes")
    _same_device(dev, w=w, bias=bias, s0=s0, dy=dy, dst=dst, workspace=ws, **out)
    _call(dev, "kda_conv_bwd", px, ld, _dense(w, "w", (D, W), torch.float32), _dense(bias, "bias", (D,), torch.float32),
          _dense(s0, "s0", (N, W - 1, D), x.dtype), _dense(dy, "dy", (B, T, D), dy.dtype), gt,
          _dense(dst, "dst", (N, W - 1, D), x.dtype), _dense(out["dx"], "dx", (B, T, D), x.dtype),
          _dense(out["dw"], "dw", (D, W), torch.float32), _dense(out.get("dbias"), "dbias", (D,), torch.float32),
          _dense(out.get("ds0"), "ds0", (N, W - 1, D), x.dtype), KDA_CONV_SILU if silu else 0, dt, B, T, D, W, arr, N,
          _ptr(ws), ws.numel())
    return out


def _qk_setup(q, k, cos, sin, pos, pos0, mode, interleaved):
    """Checked common arguments of the head norms: pointers, sizes and flags."""
    B, T, Hq, d = q.shape
    Hk = 0 if k is None else k.shape[2]
    if not -_INT_MAX <= pos0 <= _INT_MAX or cos is not None and cos.numel() > _INT_MAX and cos.shape[0] > _INT_MAX:
        raise ValueError("positions must be in 32 bits")
    if k is not None and k.dtype != q.dtype:
        raise TypeError(f"k dtype {k.dtype} != q dtype {q.dtype}")
    if mode not in ("l2", "rms"):
        raise ValueError("mode must be 'l2' or 'rms'")
    pq, ldq = _rows(q, "q", (B, T), (Hq, d))
    pk, ldk = (None, 0) if k is None else _rows(k, "k", (B, T), (Hk, d))
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin go together")
    if cos is not None and cos.dim() != 2:
        raise ValueError(f"cos must be [n_pos, rot/2], got {list(cos.shape)}")
    rot, n_pos = (0, 0) if cos is None else (2 * cos.shape[1], cos.shape[0])
    dev = q.device
    _same_device(dev, k=k)
    cos = _dense(cos, "cos", (n_pos, rot // 2), torch.float32, dev)
    sin = _dense(sin, "sin", (n_pos, rot // 2), torch.float32, dev)
    pos = _dense(pos, "pos", (B, T), torch.int32, dev) if rot else None
    flags = (KDA_QK_RMS if mode == "rms" else 0) | (KDA_QK_INTERLEAVED if interleaved else 0)
    return (pq, ldq, pk, ldk), (cos, sin, pos, int(pos0), n_pos), (flags, _dtype_code(q), B, T, Hq, Hk, d, rot)


def qk_norm_rope(q, k, wq=None, wk=None, *, cos=None, sin=None, pos=None, pos0=0, mode="l2", interleaved=False, eps=1e-6,
                 out=None):
    """qo, ko = qk_norm_rope(q, k, wq, wk): norms of the query and key heads
    with the position rotation (kda_qk_norm_rope).  q [B,T,Hq,d], k [B,T,Hk,d]
    or None (bf16 or fp32, may be slices of wider tensors); wq, wk [d] fp32 or
    None.  mode 'l2': rows divided by sqrt(sum x^2 + eps); 'rms': by
    sqrt(mean x^2 + eps).  cos, sin [n_pos, rot/2] fp32 turn the first rot
    channels (pairs (i, i+rot/2), or neighbours if interleaved) by the row
    pos [B,T] int32 gives, or pos0 + t; None: no rotation.  out: (qo, ko)
    to write to, which may be contiguous q and k themselves."""
    rows, table, sizes = _qk_setup(q, k, cos, sin, pos, pos0, mode, interleaved)
    _, _, B, T, Hq, Hk, d, _ = sizes
    dev = q.device
    qo, ko = (None, None) if out is None else out
    qo = _given(qo, q, "out[0]")
    ko = None if k is None else _given(ko, k, "out[1]")
    _call(dev, "kda_qk_norm_rope", *rows, _dense(wq, "wq", (d,), torch.float32, dev), _dense(wk, "wk", (d,), torch.float32, dev), *table,
          float(eps), qo.data_ptr(), None if ko is None else ko.data_ptr(), *sizes)
    return qo, ko


def qk_norm_rope_bwd(q, k, dqo, dko, wq=None, wk=None, *, cos=None, sin=None, pos=None, pos0=0, mode="l2", interleaved=False,
                     eps=1e-6, workspace=None, out=None):
    """Gradients of qk_norm_rope (kda_qk_norm_rope_bwd) from dqo [B,T,Hq,d] and
    dko (q's type or fp32): a dict of dq, dk (q's type) and dwq, dwk [d] fp32
    (None without that weight).  `out` may supply that dict."""
    rows, table, sizes = _qk_setup(q, k, cos, sin, pos, pos0, mode, interleaved)
    _, _, B, T, Hq, Hk, d, _ = sizes
    dev = q.device
    if k is not None and (dko is None or dko.dtype != dqo.dtype):
        raise TypeError("dqo and dko must have one type")
    if out is None:
        out = {"dq": torch.empty((B, T, Hq, d), dtype=q.dtype, device=dev),
               "dk": torch.empty((B, T, Hk, d), dtype=q.dtype, device=dev) if k is not None else None,
               "dwq": torch.empty(d, dtype=torch.float32, device=dev) if wq is not None else None,
               "dwk": torch.empty(d, dtype=torch.float32, device=dev) if wk is not None and k is not None else None}
    nbytes = lib().kda_qk_bwd_workspace_bytes(B, T, Hq, Hk, d)
    wanted = out.get("dwq") is not None or out.get("dwk") is not None
    ws = _scratch(workspace, nbytes, dev, "kda_qk_bwd_workspace_bytes") if wanted else None
    _same_device(dev, wq=wq, wk=wk, dqo=dqo, dko=dko, workspace=ws, **out)
    _call(dev, "kda_qk_norm_rope_bwd", *rows, _dense(wq, "wq", (d,), torch.float32), _dense(wk, "wk", (d,), torch.float32), *table,
          float(eps), _dense(dqo, "dqo", (B, T, Hq, d), dqo.dtype), _dense(dko if k is not None else None, "dko", (B, T, Hk, d), dqo.dtype),
          _dtype_code(dqo), _dense(out["dq"], "dq", (B, T, Hq, d), q.dtype),
          _dense(out["dk"] if k is not None else None, "dk", (B, T, Hk, d), q.dtype),
          _dense(out.get("dwq"), "dwq", (d,), torch.float32), _dense(out.get("dwk"), "dwk", (d,), torch.float32), *sizes,
          _ptr(ws), 0 if ws is None else ws.numel())
    return out


def _ssm_setup(x, dt, A, Bm, Cm, D, dt_bias, lead):
    """Checked inputs of the scan: (x .. dt_bias of the C call, G, dk)."""
    H, dv = x.shape[-2:]
    G, dk = Bm.shape[-2:]
    for n, t in (("dt", dt), ("Bm", Bm), ("Cm", Cm)):
        if t.dtype != x.dtype:
            raise TypeError(f"{n} dtype {t.dtype} != x dtype {x.dtype}")
    dev = x.device
    _same_device(dev, dt=dt, Bm=Bm, Cm=Cm)
    vec = lambda t, n: _dense(t, n, (H,), torch.float32, dev)
    return (*_rows(x, "x", lead, (H, dv)), *_rows(dt, "dt", lead, (H,)), vec(A, "A"), *_rows(Bm, "Bm", lead, (G, dk)),
            *_rows(Cm, "Cm", lead, (G, dk)), vec(D, "D"), vec(dt_bias, "dt_bias")), G, dk


def ssm_fwd_chunked(x, dt, A, Bm, Cm, h0=None, *, D=None, dt_bias=None, softplus=False, cu_seqlens=None, final_state=True, ht=None,
                    workspace=None, out=None):
    """y, ht = ssm_fwd_chunked(x, dt, A, Bm, Cm, h0): state space scan of
    prompts (kda_ssm_fwd_chunked), S_t = exp(dt A) S_{t-1} + dt B x^T, y = S^T C
    + D x.  x [B,T,H,dv], dt [B,T,H], Bm, Cm [B,T,G,dk] (bf16 or fp32, may be
    slices of wider tensors; G divides H); A, D, dt_bias [H] fp32; h0 / ht
    [N,H,dk,dv] fp32 of the N = B sequences, or of those cu_seqlens (host ints)
    cuts the packed axis into; ht may be h0 itself.  softplus: dt =
    Softplus(dt + dt_bias)."""
    B, T, H, dv = x.shape
    args, G, dk = _ssm_setup(x, dt, A, Bm, Cm, D, dt_bias, (B, T))
    arr, N = _packed(cu_seqlens, B, T)
    code, dev, st = _dtype_code(x), x.device, (N, H, dk, dv)
    y = _given(out, x, "out")
    if final_state and ht is None:
        ht = torch.empty(st, dtype=torch.float32, device=dev)
    n = lib().kda_ssm_workspace_bytes(B, T, H, dk, dv, code)
    ws = _scratch(workspace, n, dev, "kda_ssm_workspace_bytes") if n else None
    _same_device(dev, h0=h0, ht=ht, workspace=ws)
    _call(dev, "kda_ssm_fwd_chunked", *args, _dense(h0, "h0", st, torch.float32),
          _dense(ht if final_state else None, "ht", st, torch.float32), y.data_ptr(), KDA_SSM_SOFTPLUS if softplus else 0, code, B, T,
          H, G, dk, dv, arr, N, _ptr(ws), 0 if ws is None else ws.numel())
    return y, (ht if final_state else None)


def ssm_step(x, dt, A, Bm, Cm, state, *, D=None, dt_bias=None, softplus=False, state_out=None, out=None):
    """y = ssm_step(x, dt, A, Bm, Cm, state): one token per sequence
    (kda_ssm_step), x [B,H,dv], dt [B,H], Bm, Cm [B,G,dk]; state [B,H,dk,dv]
    fp32 moves on in place, or into state_out (the old state is then kept)."""
    B, H, dv = x.shape
    args, G, dk = _ssm_setup(x, dt, A, Bm, Cm, D, dt_bias, (B,))
    so = state if state_out is None else state_out
    y = _given(out, x, "out")
    dev, st = x.device, (B, H, dk, dv)
    _call(dev, "kda_ssm_step", *args, _dense(state, "state", st, torch.float32, dev),
          _dense(so, "state_out", st, torch.float32, dev), y.data_ptr(), KDA_SSM_SOFTPLUS if softplus else 0, _dtype_code(x), B,
          H, G, dk, dv)
    return y


def ssm_bwd_chunked(x, dt, A, Bm, Cm, dy, h0=None, dht=None, *, D=None, dt_bias=None, softplus=False, cu_seqlens=None, workspace=None,
                    out=None):
    """Gradients of ssm_fwd_chunked (kda_ssm_bwd_chunked) from dy [B,T,H,dv]
    (x's type) and dht [N,H,dk,dv] fp32 (gradient of ht, or None): a dict of
    dx, ddt, dB, dC (x's type) and dA, dD, ddt_bias [H], dh0 [N,H,dk,dv] fp32
    (None for an input that was not given).  `out` may supply that dict."""
    B, T, H, dv = x.shape
    args, G, dk = _ssm_setup(x, dt, A, Bm, Cm, D, dt_bias, (B, T))
    arr, N = _packed(cu_seqlens, B, T)
    code, dev, st = _dtype_code(x), x.device, (N, H, dk, dv)
    shapes = {"dx": (B, T, H, dv), "ddt": (B, T, H), "dB": (B, T, G, dk), "dC": (B, T, G, dk)}
    small = {"dA": ((H,), A), "dD": ((H,), D), "ddt_bias": ((H,), dt_bias), "dh0": (st, h0)}
    if out is None:
        out = {n: torch.empty(s, dtype=x.dtype, device=dev) for n, s in shapes.items()}
        out.update({n: torch.empty(s, dtype=torch.float32, device=dev) if t is not None else None for n, (s, t) in small.items()})
    ws = _scratch(workspace, lib().kda_ssm_bwd_workspace_bytes(B, T, H, G, dk, dv, code, N if arr is not None else 0), dev,
                  "kda_ssm_bwd_workspace_bytes")
    _same_device(dev, dy=dy, h0=h0, dht=dht, workspace=ws, **out)
    p = {n: _dense(out[n], n, s, x.dtype) for n, s in shapes.items()}
    p.update({n: _dense(out.get(n), n, s, torch.float32) for n, (s, _) in small.items()})
    _call(dev, "kda_ssm_bwd_chunked", *args, _dense(h0, "h0", st, torch.float32), _dense(dy, "dy", (B, T, H, dv), x.dtype),
          _dense(dht, "dht", st, torch.float32), p["dx"], p["ddt"], p["dA"], p["dB"], p["dC"], p["dD"], p["ddt_bias"], p["dh0"],
          KDA_SSM_SOFTPLUS if softplus else 0, code, B, T, H, G, dk, dv, arr, N, _ptr(ws), ws.numel())
    return out


# ---------------------------------------------------------------- a recurrent block's norm, projection and recurrence
def _flat_rows(t, name, D):
    """Pointer, row stride and leading sizes of rows [..., D]: one or two
    leading dimensions, as for _rows."""
    shape = t.shape
    if not 2 <= len(shape) <= 3 or shape[-1] != D:
        raise ValueError(f"{name} must be [rows, {D}] or [B, T, {D}], got {list(shape)}")
    lead = shape[:-1]
    if D <= _INT_MAX and t.is_cuda and t.is_contiguous():
        return t.data_ptr(), D, lead
    p, ld = _rows(t, name, tuple(lead), (D,))
    return p, ld, lead


def _rows_beside(t, name, dtype, dev, shape, D):
    """Pointer and token stride of rows of D of this (checked) shape, type and
    device, or of None."""
    if t is None:
        return None, 0
    if t.dtype is not dtype:
        raise TypeError(f"{name} dtype {t.dtype} != {dtype}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, not on {dev}")
    if t.shape == shape and t.is_contiguous():
        return t.data_ptr(), D
    return _rows(t, name, tuple(shape[:-1]), (D,))


def add_rms_norm(x, res=None, w=None, *, eps=1e-6, fp8=False, out=None, scale_out=None, sum_out=None):
    """y, h = add_rms_norm(x, res, w): norm of the residual stream with the
    residual's addition (kda_add_rms_norm), h = x + res in res's type (x's, or
    fp32 for a stream kept in 32 bits; None: h = x, returned as None), y =
    w h / sqrt(mean h^2 + eps) in x's type.  x, res [rows,D] or [B,T,D] (bf16 or
    fp32, may be slices of wider tensors); w [D] fp32 or None.  sum_out may be
    a contiguous res itself.  fp8: y is the pair (y8, scale): y8 in
    torch.float8_e4m3fn, scale [..., ceil(D/128)] fp32 with n = y8 scale."""
    shape = x.shape
    D = shape[-1]
    px, ldx, lead = _flat_rows(x, "x", D)
    dev, dt = x.device, _dtype_code(x)
    pr, ldr, rdt, ph = None, 0, dt, None
    if res is not None:
        pr, ldr = _rows_beside(res, "res", res.dtype, dev, shape, D)
        rdt = _dtype_code(res)
        if sum_out is None:
            sum_out = torch.empty_like(res, memory_format=torch.contiguous_format)
            ph = sum_out.data_ptr()
        else:
            ph = _dense(sum_out, "sum_out", shape, res.dtype, dev)
    elif sum_out is not None:
        raise ValueError("sum_out needs res")
    ps = None
    if fp8:
        kb = (*lead, (D + 127) // 128)
        if out is None:
            out = torch.empty_like(x, dtype=torch.float8_e4m3fn, memory_format=torch.contiguous_format)
            py = out.data_ptr()
        else:
            py = _dense(out, "out", shape, torch.float8_e4m3fn, dev)
        if scale_out is None:
            scale_out = torch.empty(kb, dtype=torch.float32, device=dev)
            ps = scale_out.data_ptr()
        else:
            ps = _dense(scale_out, "scale_out", kb, torch.float32, dev)
    else:
        out = _given(out, x, "out")
        py = out.data_ptr()
    _call(dev, "kda_add_rms_norm", px, ldx, pr, ldr, rdt, _dense(w, "w", (D,), torch.float32, dev), eps, ph, py, ps, dt, math.prod(lead), D)
    return ((out, scale_out) if fp8 else out), (None if res is None else sum_out)


def add_rms_norm_bwd(h, w, dy, dh=None, *, eps=1e-6, want_dw=None, workspace=None, out=None):
    """Gradients of add_rms_norm (kda_add_rms_norm_bwd) from h [rows,D] or
    [B,T,D] (the sum it returned, or its x), dy (bf16 or fp32) and dh (h's type,
    the gradient that reaches h past the norm, or None): a dict of dx (h's type;
    the gradient of x and of res) and dw [D] fp32 (None without w; want_dw=True:
    that of a weight of ones).  `out` may supply that dict; its dx may be dh."""
    D = h.shape[-1]
    ph, ldh, lead = _flat_rows(h, "h", D)
    dev, rows = h.device, math.prod(lead)
    if out is None:
        wanted = w is not None if want_dw is None else want_dw
        dx, dw = _given(None, h, "dx"), torch.empty(D, dtype=torch.float32, device=dev) if wanted else None
        out = {"dx": dx, "dw": dw}
        pdx, pdw = dx.data_ptr(), dw.data_ptr() if wanted else None
    else:
        pdx, pdw = _dense(out["dx"], "dx", h.shape, h.dtype, dev), _dense(out.get("dw"), "dw", (D,), torch.float32, dev)
    pws, nws = None, 0
    if pdw is not None:
        ws = _scratch(workspace, lib().kda_add_rms_norm_bwd_workspace_bytes(rows, D), dev, "kda_add_rms_norm_bwd_workspace_bytes")
        _same_device(dev, workspace=ws)
        pws, nws = _ptr(ws), ws.numel()
    _call(dev, "kda_add_rms_norm_bwd", ph, ldh, _dense(w, "w", (D,), torch.float32, dev), eps, _dense(dy, "dy", h.shape, dy.dtype, dev),
          _dtype_code(dy), _dense(dh, "dh", h.shape, h.dtype, dev), pdx, pdw, _dtype_code(h), rows, D, pws, nws)
    return out


def gemm_fp8(a, sa, w, sw, *, out_dtype=torch.bfloat16, out=None):
    """c = gemm_fp8(a, sa, w, sw): product of 8-bit rows a [M,K] or [B,T,K] and
    weights w [N,K] (torch.float8_e4m3fn; a may be a slice of a wider tensor)
    with fp32 scales sa [..., ceil(K/128)] and sw [ceil(N/128), ceil(K/128)]
    (kda_gemm_fp8): c [..., N] of out_dtype (bf16 or fp32), sums in fp32."""
    if a.dtype is not torch.float8_e4m3fn:
        raise TypeError(f"a must be torch.float8_e4m3fn, got {a.dtype}")
    if w.dtype is not torch.float8_e4m3fn:
        raise TypeError(f"w must be torch.float8_e4m3fn, got {w.dtype}")
    if sa.dtype is not torch.float32:
        raise TypeError(f"sa must be torch.float32, got {sa.dtype}")
    wshape = w.shape
    N, K = wshape
    if N > _INT_MAX or K > _INT_MAX:
        raise ValueError(f"w: a size is not in 32 bits: {list(wshape)}")
    kb = (K + 127) // 128
    pa, lda, lead = _flat_rows(a, "a", K)
    dev = a.device
    ps, lsa = _rows_beside(sa, "sa", torch.float32, dev, (*lead, kb), kb)
    if out is None:
        out = torch.empty((*lead, N), dtype=out_dtype, device=dev)
        pc = out.data_ptr()
    else:
        pc = _dense(out, "out", (*lead, N), out.dtype, dev)
    _call(dev, "kda_gemm_fp8", pa, lda, ps, lsa, _dense(w, "w", wshape, torch.float8_e4m3fn, dev),
          _dense(sw, "sw", ((N + 127) // 128, kb), torch.float32, dev), pc, _dtype_code(out), math.prod(lead), N, K)
    return out


def _lru_setup(x, r, i, c):
    """Checked inputs of the gated linear recurrence: (x .. c of the C call)."""
    shape, dev, dtype = x.shape, x.device, x.dtype
    D = shape[-1]
    pr, ldr = _rows_beside(r, "r", dtype, dev, shape, D)
    pi, ldi = _rows_beside(i, "i", dtype, dev, shape, D)
    if x.is_contiguous() and x.is_cuda and x.numel() <= _INT_MAX:
        px, ldx = x.data_ptr(), D
    else:
        px, ldx = _rows(x, "x", tuple(shape[:-1]), (D,))
    return px, ldx, pr, ldr, pi, ldi, _dense(c, "c", (D,), torch.float32, dev)


def lru_fwd(x, r, i=None, c=None, h0=None, *, unit=True, cu_seqlens=None, final_state=True, ht=None, workspace=None, out=None):
    """y, ht = lru_fwd(x, r, i, c, h0): gated linear recurrence with one state a
    channel (kda_lru_fwd), h_t = exp(g) h_{t-1} + m Sigmoid(i) x, y = h, with
    g = -c Sigmoid(r) (c None: r is the log-decay itself), m = sqrt(1 - exp(2 g))
    (unit=False: 1).  x, r, i [B,T,D] (bf16 or fp32, may be slices of wider
    tensors; i None: no input gate); c [D] fp32; h0 / ht [N,D] fp32 of the N = B
    sequences, or of those cu_seqlens (host ints) cuts the packed axis into; ht
    may be h0 itself."""
    B, T, D = x.shape
    args = _lru_setup(x, r, i, c)
    arr, N = _packed(cu_seqlens, B, T)
    dev, st = x.device, (N, D)
    y = _given(out, x, "out")
    pht = None
    if final_state:
        if ht is None:
            ht = torch.empty(st, dtype=torch.float32, device=dev)
            pht = ht.data_ptr()
        else:
            pht = _dense(ht, "ht", st, torch.float32, dev)
    ws = _scratch(workspace, lib().kda_lru_workspace_bytes(B, T, D, N if arr is not None else 0), dev, "kda_lru_workspace_bytes")
    _same_device(dev, workspace=ws)
    _call(dev, "kda_lru_fwd", *args, _dense(h0, "h0", st, torch.float32, dev), pht, y.data_ptr(),
          KDA_LRU_UNIT if unit else 0, _dtype_code(x), B, T, D, arr, N, _ptr(ws), ws.numel())
    return y, (ht if final_state else None)


def lru_step(x, r, i, c, state, *, unit=True, state_out=None, out=None):
    """y = lru_step(x, r, i, c, state): one token x, r, i [B,D] per sequence
    (kda_lru_step); state [B,D] fp32 moves on in place, or into state_out (the
    old state is then kept)."""
    st = x.shape
    B, D = st
    args = _lru_setup(x, r, i, c)
    dev = x.device
    ps = _dense(state, "state", st, torch.float32, dev)
    po = ps if state_out is None else _dense(state_out, "state_out", st, torch.float32, dev)
    y = _given(out, x, "out")
    _call(dev, "kda_lru_step", *args, ps, po, y.data_ptr(), KDA_LRU_UNIT if unit else 0, _dtype_code(x), B, D)
    return y


def lru_bwd(x, r, i, c, dy, h0=None, dht=None, *, unit=True, cu_seqlens=None, workspace=None, out=None):
    """Gradients of lru_fwd (kda_lru_bwd) from dy [B,T,D] (x's type) and dht
    [N,D] fp32 (gradient of ht, or None): a dict of dx, dr, di (x's type; di
    None without i), dc [D] fp32 (None without c) and dh0 [N,D] fp32 (None
    without h0).  `out` may supply that dict to be filled in place."""
    B, T, D = x.shape
    args = _lru_setup(x, r, i, c)
    arr, N = _packed(cu_seqlens, B, T)
    dev, st = x.device, (N, D)
    if out is None:
        out = {n: _given(None, x, n) if t is not None else None for n, t in (("dx", x), ("dr", r), ("di", i))}
        out["dc"] = torch.empty(D, dtype=torch.float32, device=dev) if c is not None else None
        out["dh0"] = torch.empty(st, dtype=torch.float32, device=dev) if h0 is not None else None
        ps = [t if t is None else t.data_ptr() for t in out.values()]
    else:
        ps = [_dense(out.get(n), n, (B, T, D), x.dtype, dev) for n in ("dx", "dr", "di")]
        ps += [_dense(out.get("dc"), "dc", (D,), torch.float32, dev), _dense(out.get("dh0"), "dh0", st, torch.float32, dev)]
    ws = _scratch(workspace, lib().kda_lru_bwd_workspace_bytes(B, T, D, N if arr is not None else 0), dev, "kda_lru_bwd_workspace_bytes")
    _same_device(dev, workspace=ws)
    _call(dev, "kda_lru_bwd", *args, _dense(h0, "h0", st, torch.float32, dev), _dense(dy, "dy", (B, T, D), x.dtype, dev),
          _dense(dht, "dht", st, torch.float32, dev), *ps, KDA_LRU_UNIT if unit else 0, _dtype_code(x), B, T, D, arr, N, _ptr(ws), ws.numel())
    return out


def stamps_read():
    """kda_stamps_read: the fused prefill's cycle stamps of the last launch,
    numpy uint64 [STAMP_WGS, STAMP_WAVES, STAMP_SLOTS] (layout in
    include/kda_stamps.h).  Only the profiling build libkda_stamps.so has
    them."""
    import numpy as np

    L = lib()
    if not hasattr(L, "kda_stamps_read"):
        raise RuntimeError(f"{LIB_PATH.name} has no cycle stamps: set kda.LIB_PATH = kda.STAMPS_LIB_PATH "
                           "before the first call")
    buf = np.zeros((STAMP_WGS, STAMP_WAVES, STAMP_SLOTS), dtype=np.uint64)
    _check(L.kda_stamps_read(buf.ctypes.data, buf.size), "kda_stamps_read")
    return buf
