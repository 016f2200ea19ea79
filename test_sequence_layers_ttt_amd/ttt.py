"""Python binding of libttt_amd.so (the C ABI in include/ttt.h).

Argument marshalling only: torch provides device memory and the stream; every
step of the scan runs in the library's HIP kernels.  There is no fallback: if
the library is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Tuple

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libttt_amd.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_LAUNCH = 0, -1, -2, -3, -4
DTYPE_F32, DTYPE_BF16 = 0, 1
PLAN_AUTO, PLAN_GENERIC, PLAN_MFMA, PLAN_BIGCHUNK, PLAN_SPLIT = 0, 1, 2, 3, 4
READ_INCLUSIVE, READ_CHUNK_START = 0, 1

# every symbol include/ttt.h declares
EXPORTS = ("ttt_linear_workspace_bytes", "ttt_linear_workspace_bytes_ex",
           "ttt_linear_select_plan", "ttt_linear_fwd",
           "ttt_linear_step", "ttt_linear_bwd_workspace_bytes", "ttt_linear_bwd",
           "ttt_linear_fwd_ex", "ttt_linear_select_plan_ex",
           "ttt_linear_fwd_varlen", "ttt_linear_select_plan_varlen", "ttt_linear_ln_fwd",
           "ttt_linear_fwd_momentum", "ttt_linear_fwd_noalloc",
           "ttt_linear_noalloc_scratch_bytes",
           "ttt_mlp_workspace_bytes", "ttt_mlp_workspace_bytes_ex", "ttt_mlp_select_plan",
           "ttt_mlp_fwd", "ttt_mlp_fwd_ex",
           "ttt_gated_workspace_bytes", "ttt_gated_fwd", "ttt_gated_step", "ttt_gated_bwd",
           "ttt_rmsnorm_fwd", "ttt_rmsnorm_q8_fwd", "ttt_rmsnorm_bwd",
           "ttt_rmsnorm_bwd_workspace_bytes", "ttt_clip_grad_norm", "ttt_clip_workspace_bytes",
           "ttt_status_string", "ttt_plan_name")


class TTTError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__("%s: %s (status %d)" % (what, status_string(status), status))
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    """Load libttt_amd.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libttt_amd.so is not built (run __graft_entry__.build()); "
                               "the TTT scan has no CPU fallback")
        L = ctypes.CDLL(LIB_PATH)
        vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        L.ttt_linear_workspace_bytes.argtypes = [i] * 5
        L.ttt_linear_workspace_bytes.restype = sz
        L.ttt_linear_workspace_bytes_ex.argtypes = [i] * 7
        L.ttt_linear_workspace_bytes_ex.restype = sz
        L.ttt_linear_select_plan.argtypes = [i] * 7
        L.ttt_linear_select_plan.restype = i
        L.ttt_linear_fwd.argtypes = [vp, vp, vp, vp, f, vp, vp, vp, i, i, i, i, i, i, vp, sz, vp]
        L.ttt_linear_fwd.restype = i
        L.ttt_linear_fwd_ex.argtypes = [vp, vp, vp, vp, f, vp, vp, vp, i, i, i, i, i, i, vp, sz,
                                        vp, i, i]
        L.ttt_linear_fwd_ex.restype = i
        L.ttt_linear_fwd_noalloc.argtypes = [vp, vp, vp, vp, f, vp, vp, vp, i, i, i, i, i, i, vp]
        L.ttt_linear_fwd_noalloc.restype = i
        L.ttt_linear_noalloc_scratch_bytes.argtypes = []
        L.ttt_linear_noalloc_scratch_bytes.restype = sz
        L.ttt_linear_fwd_momentum.argtypes = [vp, vp, vp, vp, f, vp, vp, f, vp, vp, vp,
                                              i, i, i, i, i, i, vp, sz, vp, i]
        L.ttt_linear_fwd_momentum.restype = i
        L.ttt_linear_ln_fwd.argtypes = [vp, vp, vp, vp, f, vp, vp, vp, vp, f, vp, vp, vp,
                                        i, i, i, i, i, i, vp]
        L.ttt_linear_ln_fwd.restype = i
        L.ttt_linear_fwd_varlen.argtypes = [vp, vp, vp, vp, f, vp, vp, vp, vp, i, i, i, i, i, i,
                                            vp, i]
        L.ttt_linear_fwd_varlen.restype = i
        L.ttt_linear_select_plan_varlen.argtypes = [i] * 7
        L.ttt_linear_select_plan_varlen.restype = i
        L.ttt_linear_select_plan_ex.argtypes = [i] * 8
        L.ttt_linear_select_plan_ex.restype = i
        L.ttt_linear_bwd_workspace_bytes.argtypes = [i] * 6
        L.ttt_linear_bwd_workspace_bytes.restype = sz
        L.ttt_linear_bwd.argtypes = [vp, vp, vp, vp, f, vp, vp, vp, vp, vp, vp, vp, vp,
                                     i, i, i, i, i, i, vp, sz, vp]
        L.ttt_linear_bwd.restype = i
        L.ttt_linear_step.argtypes = [vp, vp, vp, vp, f, vp, vp, i, vp, i, i, i, i, i, i, vp]
        L.ttt_linear_step.restype = i
        L.ttt_mlp_workspace_bytes.argtypes = [i] * 5
        L.ttt_mlp_workspace_bytes.restype = sz
        L.ttt_mlp_workspace_bytes_ex.argtypes = [i] * 7
        L.ttt_mlp_workspace_bytes_ex.restype = sz
        L.ttt_mlp_select_plan.argtypes = [i] * 7
        L.ttt_mlp_select_plan.restype = i
        L.ttt_mlp_fwd.argtypes = [vp, vp, vp, vp, f, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                  i, i, i, i, i, i, vp, sz, vp]
        L.ttt_mlp_fwd.restype = i
        L.ttt_mlp_fwd_ex.argtypes = [vp, vp, vp, vp, f, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                     i, i, i, i, i, i, vp, sz, vp, i]
        L.ttt_mlp_fwd_ex.restype = i
        ll = ctypes.c_longlong
        L.ttt_gated_workspace_bytes.argtypes = [i] * 5
        L.ttt_gated_workspace_bytes.restype = sz
        L.ttt_gated_fwd.argtypes = [vp] * 5 + [i] * 5 + [vp, sz, vp]
        L.ttt_gated_fwd.restype = i
        L.ttt_gated_step.argtypes = [vp] * 4 + [i] * 5 + [vp]
        L.ttt_gated_step.restype = i
        L.ttt_gated_bwd.argtypes = [vp] * 8 + [i] * 5 + [vp, sz, vp]
        L.ttt_gated_bwd.restype = i
        L.ttt_rmsnorm_fwd.argtypes = [vp, vp, vp, f, vp, vp, ll, i, i, vp]
        L.ttt_rmsnorm_fwd.restype = i
        L.ttt_rmsnorm_q8_fwd.argtypes = [vp, vp, vp, f, vp, vp, vp, ll, i, i, vp]
        L.ttt_rmsnorm_q8_fwd.restype = i
        L.ttt_rmsnorm_bwd.argtypes = [vp, vp, vp, vp, f, vp, vp, ll, i, i, vp, sz, vp]
        L.ttt_rmsnorm_bwd.restype = i
        L.ttt_rmsnorm_bwd_workspace_bytes.argtypes = [ll, i, i]
        L.ttt_rmsnorm_bwd_workspace_bytes.restype = sz
        L.ttt_clip_grad_norm.argtypes = [i, vp, vp, vp, vp, f, f, vp, vp, sz, vp]
        L.ttt_clip_grad_norm.restype = i
        L.ttt_clip_workspace_bytes.argtypes = []
        L.ttt_clip_workspace_bytes.restype = sz
        L.ttt_status_string.argtypes = [i]
        L.ttt_status_string.restype = ctypes.c_char_p
        L.ttt_plan_name.argtypes = [i]
        L.ttt_plan_name.restype = ctypes.c_char_p
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().ttt_status_string(int(status)).decode()


def plan_name(plan: int) -> str:
    return lib().ttt_plan_name(int(plan)).decode()


_INT_MAX = 0x7fffffff


def _fits(*sizes):
    """Refuses what the library's int arguments cannot hold: ctypes would drop the upper bits."""
    for n in sizes:
        if not -_INT_MAX - 1 <= n <= _INT_MAX:
            raise ValueError("a size of %d is beyond the library's 32 bits" % n)


def _io_dtype(t) -> int:
    import torch
    if t.dtype == torch.float32:
        return DTYPE_F32
    if t.dtype == torch.bfloat16:
        return DTYPE_BF16
    raise TypeError("K/Q/V must be float32 or bfloat16, got %s" % t.dtype)


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(device, stream) -> int:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream


def _check(t, name, shape, dtype=None):
    import torch
    if t is None:
        raise ValueError("%s is required" % name)
    _fits(*t.shape)
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s" % (name, dtype))


def linear_workspace_bytes(B, H, T, d, chunk, io_dtype=None, plan=PLAN_AUTO) -> int:
    """Workspace bytes for the shape; with io_dtype, for that dtype and plan exactly."""
    _fits(B, H, T, d, chunk)
    if io_dtype is None:
        return int(lib().ttt_linear_workspace_bytes(B, H, T, d, chunk))
    return int(lib().ttt_linear_workspace_bytes_ex(B, H, T, d, chunk, io_dtype, plan))


def linear_select_plan(B, H, T, d, chunk, io_dtype, plan=PLAN_AUTO,
                       read_mode: int = READ_INCLUSIVE) -> int:
    _fits(B, H, T, d, chunk)
    if read_mode == READ_INCLUSIVE:
        return int(lib().ttt_linear_select_plan(B, H, T, d, chunk, io_dtype, plan))
    return int(lib().ttt_linear_select_plan_ex(B, H, T, d, chunk, io_dtype, plan, read_mode))


def mlp_workspace_bytes(B, H, T, d, chunk, io_dtype=None, plan=PLAN_AUTO) -> int:
    """Workspace bytes for the shape; with io_dtype, for that dtype and plan exactly."""
    _fits(B, H, T, d, chunk)
    if io_dtype is None:
        return int(lib().ttt_mlp_workspace_bytes(B, H, T, d, chunk))
    return int(lib().ttt_mlp_workspace_bytes_ex(B, H, T, d, chunk, io_dtype, plan))


def mlp_select_plan(B, H, T, d, chunk, io_dtype, plan=PLAN_AUTO) -> int:
    _fits(B, H, T, d, chunk)
    return int(lib().ttt_mlp_select_plan(B, H, T, d, chunk, io_dtype, plan))


def _workspace(nbytes, device, workspace):
    import torch
    if nbytes == 0:
        return None
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return workspace


def linear_fwd(K, Q, V, eta, W0, chunk: int, eta_scalar: float = 0.0, *, Z=None, W_out=None,
               workspace=None, plan: int = PLAN_AUTO, stream=None,
               read_mode: int = READ_INCLUSIVE) -> Tuple:
    """TTT-Linear forward scan.  K, Q, V: [B, H, T, d] fp32 or bf16; eta: [B, H, T]
    fp32 or None (then eta_scalar); W0: [B, H, d, d] fp32; read_mode: READ_INCLUSIVE
    or READ_CHUNK_START.  Returns (Z, W_out)."""
    import torch
    B, H, T, d = K.shape
    _check(K, "K", (B, H, T, d))
    _check(Q, "Q", (B, H, T, d), K.dtype)
    _check(V, "V", (B, H, T, d), K.dtype)
    _check(W0, "W0", (B, H, d, d), torch.float32)
    if eta is not None:
        _check(eta, "eta", (B, H, T), torch.float32)
    if Z is None:
        Z = torch.empty_like(K)
    if W_out is None:
        W_out = torch.empty_like(W0)
    _check(Z, "Z", (B, H, T, d), K.dtype)
    _check(W_out, "W_out", (B, H, d, d), torch.float32)
    io = _io_dtype(K)
    p = linear_select_plan(B, H, T, d, chunk, io, plan, read_mode)
    nbytes = linear_workspace_bytes(B, H, T, d, chunk, io, p) if p > 0 else 0
    ws = _workspace(nbytes, K.device, workspace)
    rc = lib().ttt_linear_fwd_ex(K.data_ptr(), Q.data_ptr(), V.data_ptr(), _ptr(eta),
                                 float(eta_scalar), W0.data_ptr(), Z.data_ptr(),
                                 W_out.data_ptr(), B, H, T, d, int(chunk), io, _ptr(ws),
                                 0 if ws is None else ws.numel(), _stream(K.device, stream),
                                 int(plan), int(read_mode))
    if rc != OK:
        raise TTTError(rc, "ttt_linear_fwd")
    return Z, W_out


def linear_fwd_noalloc(K, Q, V, eta, W0, chunk: int, eta_scalar: float = 0.0, *, Z, W_out,
                       stream=None) -> Tuple:
    """ttt_linear_fwd_noalloc: the AUTO-plan scan with any workspace taken from the
    library's static per-GPU scratch.  Z and W_out are caller-given (this call
    allocates nothing).  Returns (Z, W_out)."""
    import torch
    B, H, T, d = K.shape
    _check(K, "K", (B, H, T, d))
    _check(Q, "Q", (B, H, T, d), K.dtype)
    _check(V, "V", (B, H, T, d), K.dtype)
    _check(W0, "W0", (B, H, d, d), torch.float32)
    if eta is not None:
        _check(eta, "eta", (B, H, T), torch.float32)
    _check(Z, "Z", (B, H, T, d), K.dtype)
    _check(W_out, "W_out", (B, H, d, d), torch.float32)
    _fits(chunk)
    rc = lib().ttt_linear_fwd_noalloc(K.data_ptr(), Q.data_ptr(), V.data_ptr(), _ptr(eta),
                                      float(eta_scalar), W0.data_ptr(), Z.data_ptr(),
                                      W_out.data_ptr(), B, H, T, d, int(chunk), _io_dtype(K),
                                      _stream(K.device, stream))
    if rc != OK:
        raise TTTError(rc, "ttt_linear_fwd_noalloc")
    return Z, W_out


def linear_noalloc_scratch_bytes() -> int:
    return int(lib().ttt_linear_noalloc_scratch_bytes())


def linear_bwd_workspace_bytes(B, H, T, d, chunk, io_dtype) -> int:
    _fits(B, H, T, d, chunk)
    return int(lib().ttt_linear_bwd_workspace_bytes(B, H, T, d, chunk, io_dtype))


def linear_bwd(K, Q, V, eta, W0, dZ, chunk: int, eta_scalar: float = 0.0, dW_T=None, *,
               dK=None, dQ=None, dV=None, deta=None, dW0=None, want_deta: bool = True,
               workspace=None, stream=None) -> Tuple:
    """Gradients of <dZ, Z> + <dW_T, W_T> through linear_fwd(K, Q, V, eta, W0, chunk).
    dZ: like K; dW_T: [B, H, d, d] fp32 or None.  Returns (dK, dQ, dV, deta, dW0);
    deta [B, H, T] fp32 is per token (None when want_deta is False)."""
    import torch
    B, H, T, d = K.shape
    _check(K, "K", (B, H, T, d))
    _check(Q, "Q", (B, H, T, d), K.dtype)
    _check(V, "V", (B, H, T, d), K.dtype)
    _check(dZ, "dZ", (B, H, T, d), K.dtype)
    _check(W0, "W0", (B, H, d, d), torch.float32)
    if eta is not None:
        _check(eta, "eta", (B, H, T), torch.float32)
    if dW_T is not None:
        _check(dW_T, "dW_T", (B, H, d, d), torch.float32)
    dK = torch.empty_like(K) if dK is None else dK
    dQ = torch.empty_like(K) if dQ is None else dQ
    dV = torch.empty_like(K) if dV is None else dV
    dW0 = torch.empty_like(W0) if dW0 is None else dW0
    if want_deta and deta is None:
        deta = torch.empty((B, H, T), dtype=torch.float32, device=K.device)
    for t, name in ((dK, "dK"), (dQ, "dQ"), (dV, "dV")):
        _check(t, name, (B, H, T, d), K.dtype)
    _check(dW0, "dW0", (B, H, d, d), torch.float32)
    if deta is not None:
        _check(deta, "deta", (B, H, T), torch.float32)
    io = _io_dtype(K)
    nbytes = linear_bwd_workspace_bytes(B, H, T, d, chunk, io)
    if nbytes == 0:
        raise TTTError(ERR_UNSUPPORTED, "ttt_linear_bwd")
    ws = _workspace(nbytes, K.device, workspace)
    rc = lib().ttt_linear_bwd(K.data_ptr(), Q.data_ptr(), V.data_ptr(), _ptr(eta),
                              float(eta_scalar), W0.data_ptr(), dZ.data_ptr(), _ptr(dW_T),
                              dK.data_ptr(), dQ.data_ptr(), dV.data_ptr(), _ptr(deta),
                              dW0.data_ptr(), B, H, T, d, int(chunk), io, _ptr(ws),
                              ws.numel(), _stream(K.device, stream))
    if rc != OK:
        raise TTTError(rc, "ttt_linear_bwd")
    return dK, dQ, dV, deta, dW0


def linear_step(K, Q, V, eta, W_chunk, G, pos: int, chunk: int, eta_scalar: float = 0.0, *,
                Z=None, stream=None):
    """Continue TTT-Linear scans by n tokens from a carried state, in place.
    K, Q, V: [B, H, n, d] fp32 or bf16; eta: [B, H, n] fp32 or None; W_chunk (the
    chunk-start state) and G (the chunk's update so far): [B, H, d, d] fp32, both
    updated in place; pos: tokens of the current chunk already read.  Returns
    (Z, new pos); the state after the last token is W_chunk - G."""
    import torch
    B, H, n, d = K.shape
    _check(K, "K", (B, H, n, d))
    _check(Q, "Q", (B, H, n, d), K.dtype)
    _check(V, "V", (B, H, n, d), K.dtype)
    _check(W_chunk, "W_chunk", (B, H, d, d), torch.float32)
    _check(G, "G", (B, H, d, d), torch.float32)
    if eta is not None:
        _check(eta, "eta", (B, H, n), torch.float32)
    if Z is None:
        Z = torch.empty_like(K)
    _check(Z, "Z", (B, H, n, d), K.dtype)
    _fits(pos, chunk)
    rc = lib().ttt_linear_step(K.data_ptr(), Q.data_ptr(), V.data_ptr(), _ptr(eta),
                               float(eta_scalar), W_chunk.data_ptr(), G.data_ptr(), int(pos),
                               Z.data_ptr(), B, H, n, d, int(chunk), _io_dtype(K),
                               _stream(K.device, stream))
    if rc != OK:
        raise TTTError(rc, "ttt_linear_step")
    return Z, (int(pos) + n) % int(chunk)


def linear_fwd_momentum(K, Q, V, eta, W0, Mom0, beta: float, chunk: int,
                        eta_scalar: float = 0.0, *, Z=None, W_out=None, Mom_out=None,
                        workspace=None, plan: int = PLAN_AUTO, stream=None) -> Tuple:
    """TTT-Linear with a momentum state and chunk-start reads.  Mom0: [B, H, d, d]
    fp32 or None (zero).  Returns (Z, W_out, Mom_out)."""
    import torch
    B, H, T, d = K.shape
    _check(K, "K", (B, H, T, d))
    _check(Q, "Q", (B, H, T, d), K.dtype)
    _check(V, "V", (B, H, T, d), K.dtype)
    _check(W0, "W0", (B, H, d, d), torch.float32)
    if Mom0 is not None:
        _check(Mom0, "Mom0", (B, H, d, d), torch.float32)
    if eta is not None:
        _check(eta, "eta", (B, H, T), torch.float32)
    Z = torch.empty_like(K) if Z is None else Z
    W_out = torch.empty_like(W0) if W_out is None else W_out
    Mom_out = torch.empty_like(W0) if Mom_out is None else Mom_out
    io = _io_dtype(K)
    p = linear_select_plan(B, H, T, d, chunk, io, plan, READ_CHUNK_START)
    nbytes = linear_workspace_bytes(B, H, T, d, chunk, io, p) if p > 0 else 0
    ws = _workspace(nbytes, K.device, workspace)
    rc = lib().ttt_linear_fwd_momentum(K.data_ptr(), Q.data_ptr(), V.data_ptr(), _ptr(eta),
                                       float(eta_scalar), W0.data_ptr(), _ptr(Mom0), float(beta),
                                       Z.data_ptr(), W_out.data_ptr(), Mom_out.data_ptr(),
                                       B, H, T, d, int(chunk), io, _ptr(ws),
                                       0 if ws is None else ws.numel(),
                                       _stream(K.device, stream), int(plan))
    if rc != OK:
        raise TTTError(rc, "ttt_linear_fwd_momentum")
    return Z, W_out, Mom_out


def linear_ln_fwd(K, Q, V, eta, W0, b0, ln_weight, ln_bias, chunk: int, eps: float = 1e-6,
                  eta_scalar: float = 0.0, *, Z=None, W_out=None, b_out=None,
                  stream=None) -> Tuple:
    """TTT-Linear with f(x) = x + LN(W x + b) (ln_weight, ln_bias: [H, d]) or
    f(x) = W x + b (both None).  b0: [B, H, d].  Returns (Z, W_out, b_out)."""
    import torch
    B, H, T, d = K.shape
    _check(K, "K", (B, H, T, d))
    _check(Q, "Q", (B, H, T, d), K.dtype)
    _check(V, "V", (B, H, T, d), K.dtype)
    _check(W0, "W0", (B, H, d, d), torch.float32)
    _check(b0, "b0", (B, H, d), torch.float32)
    if (ln_weight is None) != (ln_bias is None):
        raise ValueError("ln_weight and ln_bias go together")
    if ln_weight is not None:
        _check(ln_weight, "ln_weight", (H, d), torch.float32)
        _check(ln_bias, "ln_bias", (H, d), torch.float32)
    if eta is not None:
        _check(eta, "eta", (B, H, T), torch.float32)
    Z = torch.empty_like(K) if Z is None else Z
    W_out = torch.empty_like(W0) if W_out is None else W_out
    b_out = torch.empty_like(b0) if b_out is None else b_out
    _fits(chunk)
    rc = lib().ttt_linear_ln_fwd(K.data_ptr(), Q.data_ptr(), V.data_ptr(), _ptr(eta),
                                 float(eta_scalar), W0.data_ptr(), b0.data_ptr(), _ptr(ln_weight),
                                 _ptr(ln_bias), float(eps), Z.data_ptr(), W_out.data_ptr(),
                                 b_out.data_ptr(), B, H, T, d, int(chunk), _io_dtype(K),
                                 _stream(K.device, stream))
    if rc != OK:
        raise TTTError(rc, "ttt_linear_ln_fwd")
    return Z, W_out, b_out


def linear_select_plan_varlen(n_docs, H, total_T, d, chunk, io_dtype, plan=PLAN_AUTO) -> int:
    _fits(n_docs, H, total_T, d, chunk)
    return int(lib().ttt_linear_select_plan_varlen(n_docs, H, total_T, d, chunk, io_dtype, plan))


def linear_fwd_varlen(K, Q, V, eta, W0, cu_seqlens, chunk: int, eta_scalar: float = 0.0, *,
                      Z=None, W_out=None, plan: int = PLAN_AUTO, stream=None) -> Tuple:
    """TTT-Linear over packed documents, each reset to its own initial state.
    K, Q, V: [H, total_T, d]; eta: [H, total_T] or None; W0: [n_docs, H, d, d];
    cu_seqlens: int32 device tensor [n_docs + 1].  Returns (Z, W_out)."""
    import torch
    H, total_T, d = K.shape
    n_docs = cu_seqlens.numel() - 1
    _check(K, "K", (H, total_T, d))
    _check(Q, "Q", (H, total_T, d), K.dtype)
    _check(V, "V", (H, total_T, d), K.dtype)
    _check(W0, "W0", (n_docs, H, d, d), torch.float32)
    _check(cu_seqlens, "cu_seqlens", (n_docs + 1,), torch.int32)
    if eta is not None:
        _check(eta, "eta", (H, total_T), torch.float32)
    if Z is None:
        Z = torch.zeros_like(K)
    if W_out is None:
        W_out = torch.empty_like(W0)
    _check(Z, "Z", (H, total_T, d), K.dtype)
    _check(W_out, "W_out", (n_docs, H, d, d), torch.float32)
    _fits(chunk)
    rc = lib().ttt_linear_fwd_varlen(K.data_ptr(), Q.data_ptr(), V.data_ptr(), _ptr(eta),
                                     float(eta_scalar), W0.data_ptr(), Z.data_ptr(),
                                     W_out.data_ptr(), cu_seqlens.data_ptr(), n_docs, H, total_T,
                                     d, int(chunk), _io_dtype(K), _stream(K.device, stream),
                                     int(plan))
    if rc != OK:
        raise TTTError(rc, "ttt_linear_fwd_varlen")
    return Z, W_out


def mlp_fwd(K, Q, V, eta, W1, b1, W2, b2, chunk: int, eta_scalar: float = 0.0, *, Z=None,
            W1_out=None, b1_out=None, W2_out=None, b2_out=None, workspace=None,
            plan: int = PLAN_AUTO, stream=None) -> Tuple:
    """TTT-MLP forward scan (hidden 4d).  W1: [B, H, 4d, d], b1: [B, H, 4d] or None,
    W2: [B, H, d, 4d], b2: [B, H, d] or None.  Returns (Z, W1, b1, W2, b2) final."""
    import torch
    B, H, T, d = K.shape
    hd = 4 * d
    _check(K, "K", (B, H, T, d))
    _check(Q, "Q", (B, H, T, d), K.dtype)
    _check(V, "V", (B, H, T, d), K.dtype)
    _check(W1, "W1", (B, H, hd, d), torch.float32)
    _check(W2, "W2", (B, H, d, hd), torch.float32)
    if b1 is not None:
        _check(b1, "b1", (B, H, hd), torch.float32)
    if b2 is not None:
        _check(b2, "b2", (B, H, d), torch.float32)
    if eta is not None:
        _check(eta, "eta", (B, H, T), torch.float32)
    Z = torch.empty_like(K) if Z is None else Z
    W1_out = torch.empty_like(W1) if W1_out is None else W1_out
    W2_out = torch.empty_like(W2) if W2_out is None else W2_out
    if b1 is not None and b1_out is None:
        b1_out = torch.empty_like(b1)
    if b2 is not None and b2_out is None:
        b2_out = torch.empty_like(b2)
    io = _io_dtype(K)
    nbytes = mlp_workspace_bytes(B, H, T, d, chunk, io, plan)
    ws = _workspace(nbytes, K.device, workspace)
    rc = lib().ttt_mlp_fwd_ex(K.data_ptr(), Q.data_ptr(), V.data_ptr(), _ptr(eta),
                              float(eta_scalar), W1.data_ptr(), _ptr(b1), W2.data_ptr(), _ptr(b2),
                              Z.data_ptr(), W1_out.data_ptr(), _ptr(b1_out), W2_out.data_ptr(),
                              _ptr(b2_out), B, H, T, d, int(chunk), io, _ptr(ws),
                              0 if ws is None else ws.numel(), _stream(K.device, stream),
                              int(plan))
    if rc != OK:
        raise TTTError(rc, "ttt_mlp_fwd")
    return Z, W1_out, b1_out, W2_out, b2_out


# ---- operators around the scan: gated recurrence, RMS norm, gradient clipping ----
# A decoded token's call is a few microseconds of kernel, so what it checks it checks
# cheaply: the device as an index, and no context or stream object on the usual path.

def _match(t, name, shape, dtype, index):
    """_check for the operators below: on the device of that index."""
    if t.get_device() != index:
        raise ValueError("%s is on %s, expected cuda:%d" % (name, t.device, index))
    if t.dtype != dtype:
        raise ValueError("%s must be %s" % (name, dtype))
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _first(t, name):
    """Checks the tensor that the others are held to: (its ttt_dtype, its device's index)."""
    index = t.get_device()
    if index < 0:
        raise ValueError("%s must be a device tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return _io_dtype(t), index


def _elsewhere(index, stream):
    """None where a call runs on the current device and stream; else what makes them so.
    A call enters it before it allocates: a workspace that it drops then belongs to the
    stream it runs on, and is not handed to another while it still runs."""
    import torch
    if stream is not None:
        if stream.device.index != index:
            raise ValueError("the stream belongs to %s, the tensors to cuda:%d"
                             % (stream.device, index))
        return torch.cuda.stream(stream)
    return None if torch._C._cuda_getDevice() == index else torch.cuda.device(index)


def _raw_stream(index) -> int:
    """The current stream of the device (without the object that current_stream makes)."""
    import torch
    return torch._C._cuda_getCurrentRawStream(index)


def _scratch(nbytes, like, workspace):
    """_workspace for the operators below: a given one is bytes, on the tensors' device."""
    if workspace is not None:
        import torch
        if workspace.device != like.device or workspace.dtype != torch.uint8 \
                or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous uint8 tensor on %s" % like.device)
    return _workspace(nbytes, like.device, workspace)


def gated_workspace_bytes(B, H, T, d, io_dtype) -> int:
    _fits(B, H, T, d)
    return int(lib().ttt_gated_workspace_bytes(B, H, T, d, io_dtype))


def gated_fwd(X, G, h0=None, *, Z=None, h_out=None, workspace=None, stream=None) -> Tuple:
    """Gated linear recurrence h_t = exp(G_t) h_{t-1} + X_t over [B, H, T, d] fp32 or
    bf16 (G <= 0; -inf, or the type's lowest value, starts anew).  h0: [B, H, d] fp32 or None (zero).  Returns
    (Z, h_T): the states in the I/O type, and the last one in fp32."""
    import torch
    if X.numel() > _INT_MAX:       # (else no size is)
        _fits(*X.shape)
    io, dev = _first(X, "X")
    on = _elsewhere(dev, stream)
    if on is not None:
        with on:
            return gated_fwd(X, G, h0, Z=Z, h_out=h_out, workspace=workspace)
    shape = X.shape
    B, H, T, d = shape
    _match(G, "G", shape, X.dtype, dev)
    if h0 is not None:
        _match(h0, "h0", (B, H, d), torch.float32, dev)
    if Z is None:
        Z = torch.empty_like(X)
    else:
        _match(Z, "Z", shape, X.dtype, dev)
    if h_out is None:
        h_out = torch.empty((B, H, d), dtype=torch.float32, device=X.device)
    else:
        _match(h_out, "h_out", (B, H, d), torch.float32, dev)
    L = lib()
    ws = _scratch(L.ttt_gated_workspace_bytes(B, H, T, d, io), X, workspace)
    rc = L.ttt_gated_fwd(X.data_ptr(), G.data_ptr(), _ptr(h0), Z.data_ptr(), h_out.data_ptr(),
                         B, H, T, d, io, _ptr(ws), 0 if ws is None else ws.numel(),
                         _raw_stream(dev))
    if rc != OK:
        raise TTTError(rc, "ttt_gated_fwd")
    return Z, h_out


def gated_step(X, G, h, *, Z=None, stream=None):
    """Continue gated recurrences by the n tokens of X, G [B, H, n, d] from the state h
    [B, H, d] fp32, which is updated in place.  Returns Z."""
    import torch
    if X.numel() > _INT_MAX:       # (else no size is)
        _fits(*X.shape)
    io, dev = _first(X, "X")
    on = _elsewhere(dev, stream)
    if on is not None:
        with on:
            return gated_step(X, G, h, Z=Z)
    shape = X.shape
    B, H, n, d = shape
    _match(G, "G", shape, X.dtype, dev)
    _match(h, "h", (B, H, d), torch.float32, dev)
    if Z is None:
        Z = torch.empty_like(X)
    else:
        _match(Z, "Z", shape, X.dtype, dev)
    rc = lib().ttt_gated_step(X.data_ptr(), G.data_ptr(), h.data_ptr(), Z.data_ptr(), B, H, n, d,
                              io, _raw_stream(dev))
    if rc != OK:
        raise TTTError(rc, "ttt_gated_step")
    return Z


def gated_bwd(G, Z, dZ, h0=None, dh_T=None, *, dX=None, dG=None, dh0=None, workspace=None,
              stream=None) -> Tuple:
    """Gradients of <dZ, Z> + <dh_T, h_T> through Z, h_T = gated_fwd(X, G, h0).  Z is the
    forward call's; h0 and dh_T: [B, H, d] fp32 or None (zero).  Returns (dX, dG, dh0)."""
    import torch
    if G.numel() > _INT_MAX:       # (else no size is)
        _fits(*G.shape)
    io, dev = _first(G, "G")
    on = _elsewhere(dev, stream)
    if on is not None:
        with on:
            return gated_bwd(G, Z, dZ, h0, dh_T, dX=dX, dG=dG, dh0=dh0, workspace=workspace)
    shape = G.shape
    B, H, T, d = shape
    _match(Z, "Z", shape, G.dtype, dev)
    _match(dZ, "dZ", shape, G.dtype, dev)
    for t, name in ((h0, "h0"), (dh_T, "dh_T"), (dh0, "dh0")):
        if t is not None:
            _match(t, name, (B, H, d), torch.float32, dev)
    if dX is None:
        dX = torch.empty_like(G)
    else:
        _match(dX, "dX", shape, G.dtype, dev)
    if dG is None:
        dG = torch.empty_like(G)
    else:
        _match(dG, "dG", shape, G.dtype, dev)
    if dh0 is None:
        dh0 = torch.empty((B, H, d), dtype=torch.float32, device=G.device)
    L = lib()
    ws = _scratch(L.ttt_gated_workspace_bytes(B, H, T, d, io), G, workspace)
    rc = L.ttt_gated_bwd(G.data_ptr(), Z.data_ptr(), _ptr(h0), dZ.data_ptr(), _ptr(dh_T),
                         dX.data_ptr(), dG.data_ptr(), dh0.data_ptr(), B, H, T, d, io, _ptr(ws),
                         0 if ws is None else ws.numel(), _raw_stream(dev))
    if rc != OK:
        raise TTTError(rc, "ttt_gated_bwd")
    return dX, dG, dh0


def _rms_args(X, weight, residual, name="X"):
    import torch
    shape = X.shape
    if not shape or not shape[-1]:
        raise ValueError("%s needs a feature axis" % name)
    D = shape[-1]
    if D > _INT_MAX:
        _fits(D)
    io, dev = _first(X, name)
    if weight is not None:
        _match(weight, "weight", (D,), torch.float32, dev)
    if residual is not None:
        _match(residual, "residual", shape, X.dtype, dev)
    return io, dev, D, X.numel() // D


def rmsnorm_fwd(X, weight=None, residual=None, eps: float = 1e-6, *, Y=None, R=None,
                stream=None) -> Tuple:
    """RMS norm over the last axis with the residual's addition: r = X + residual,
    y = r / sqrt(mean(r^2) + eps) * weight.  X, residual: [..., D] fp32 or bf16; weight:
    [D] fp32 or None.  Returns (Y, R): R is r, or None without a residual (unless a
    tensor for it is given)."""
    import torch
    io, dev, D, rows = _rms_args(X, weight, residual)
    on = _elsewhere(dev, stream)
    if on is not None:
        with on:
            return rmsnorm_fwd(X, weight, residual, eps, Y=Y, R=R)
    if Y is None:
        Y = torch.empty_like(X)
    else:
        _match(Y, "Y", X.shape, X.dtype, dev)
    if R is not None:
        _match(R, "R", X.shape, X.dtype, dev)
    elif residual is not None:
        R = torch.empty_like(X)
    rc = lib().ttt_rmsnorm_fwd(X.data_ptr(), _ptr(residual), _ptr(weight), eps, Y.data_ptr(),
                               _ptr(R), rows, D, io, _raw_stream(dev))
    if rc != OK:
        raise TTTError(rc, "ttt_rmsnorm_fwd")
    return Y, R


def rmsnorm_q8_fwd(X, weight=None, residual=None, eps: float = 1e-6, *, Y8=None, scale=None,
                   R=None, stream=None) -> Tuple:
    """rmsnorm_fwd with y in 8-bit floating point (torch.float8_e4m3fn) and one fp32 scale
    per row: y = Y8 * scale.  Returns (Y8, scale, R)."""
    import torch
    io, dev, D, rows = _rms_args(X, weight, residual)
    on = _elsewhere(dev, stream)
    if on is not None:
        with on:
            return rmsnorm_q8_fwd(X, weight, residual, eps, Y8=Y8, scale=scale, R=R)
    if Y8 is None:
        Y8 = torch.empty_like(X, dtype=torch.float8_e4m3fn)
    else:
        _match(Y8, "Y8", X.shape, torch.float8_e4m3fn, dev)
    if scale is None:
        scale = torch.empty(X.shape[:-1], dtype=torch.float32, device=X.device)
    else:
        _match(scale, "scale", X.shape[:-1], torch.float32, dev)
    if R is not None:
        _match(R, "R", X.shape, X.dtype, dev)
    elif residual is not None:
        R = torch.empty_like(X)
    rc = lib().ttt_rmsnorm_q8_fwd(X.data_ptr(), _ptr(residual), _ptr(weight), eps, Y8.data_ptr(),
                                  scale.data_ptr(), _ptr(R), rows, D, io, _raw_stream(dev))
    if rc != OK:
        raise TTTError(rc, "ttt_rmsnorm_q8_fwd")
    return Y8, scale, R


def rmsnorm_bwd_workspace_bytes(rows, D, io_dtype) -> int:
    _fits(D)
    return int(lib().ttt_rmsnorm_bwd_workspace_bytes(rows, D, io_dtype))


def rmsnorm_bwd(R, weight, dY, dR=None, eps: float = 1e-6, *, dX=None, dweight=None,
                want_dweight: bool = True, workspace=None, stream=None) -> Tuple:
    """Gradients through rmsnorm_fwd.  R: the r it returned (X where there was no
    residual); dR: the gradient that reaches r by itself, or None.  Returns (dX, dweight):
    dX is the gradient for X and for the residual, dweight [D] fp32 (None when
    want_dweight is False)."""
    import torch
    io, dev, D, rows = _rms_args(R, weight, None, "R")
    on = _elsewhere(dev, stream)
    if on is not None:
        with on:
            return rmsnorm_bwd(R, weight, dY, dR, eps, dX=dX, dweight=dweight,
                               want_dweight=want_dweight, workspace=workspace)
    _match(dY, "dY", R.shape, R.dtype, dev)
    if dR is not None:
        _match(dR, "dR", R.shape, R.dtype, dev)
    if dX is None:
        dX = torch.empty_like(R)
    else:
        _match(dX, "dX", R.shape, R.dtype, dev)
    if dweight is not None:
        _match(dweight, "dweight", (D,), torch.float32, dev)
    elif want_dweight:
        dweight = torch.empty(D, dtype=torch.float32, device=R.device)
    L = lib()
    ws = None
    if dweight is not None:
        ws = _scratch(L.ttt_rmsnorm_bwd_workspace_bytes(rows, D, io), R, workspace)
    rc = L.ttt_rmsnorm_bwd(R.data_ptr(), _ptr(weight), dY.data_ptr(), _ptr(dR), eps,
                           dX.data_ptr(), _ptr(dweight), rows, D, io, _ptr(ws),
                           0 if ws is None else ws.numel(), _raw_stream(dev))
    if rc != OK:
        raise TTTError(rc, "ttt_rmsnorm_bwd")
    return dX, dweight


def clip_workspace_bytes() -> int:
    return int(lib().ttt_clip_workspace_bytes())


def clip_grad_norm(grads, max_norm: float, eps: float = 1e-6, *, outs=None, norm=None,
                   workspace=None, stream=None) -> Tuple:
    """The 2-norm over all tensors of the list `grads` (fp32 or bf16, any contiguous
    shapes, one device), and each of them times min(1, max_norm / (norm + eps)).  outs:
    the list of tensors to write, of the same types and numbers of elements, which may be
    grads itself (in place); None makes new ones.  Returns (outs, norm): norm is a [1] fp32 device tensor."""
    import torch
    grads = list(grads)
    n = len(grads)
    if n == 0 and norm is None:
        raise ValueError("no gradients, and no tensor for the norm")
    ref = grads[0] if n else norm
    dev = ref.get_device()
    if dev < 0:
        raise ValueError("%s must be a device tensor" % ("grads[0]" if n else "norm"))
    on = _elsewhere(dev, stream)
    if on is not None:
        with on:
            return clip_grad_norm(grads, max_norm, eps, outs=outs, norm=norm, workspace=workspace)
    # (whole lists at a time: a model has hundreds of tensors, and each check of one costs
    # as much as scaling a small one)
    tensor = torch.Tensor
    types = [g.dtype for g in grads]
    if any(map(dev.__ne__, map(tensor.get_device, grads))) \
            or not all(map(tensor.is_contiguous, grads)):
        for k, g in enumerate(grads):
            _match(g, "grads[%d]" % k, g.shape, g.dtype, dev)
    codes = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}
    kinds, sizes = [codes.get(t) for t in types], list(map(tensor.numel, grads))
    if None in kinds:
        raise TypeError("grads[%d] must be float32 or bfloat16, got %s"
                        % (kinds.index(None), types[kinds.index(None)]))
    if norm is None:
        norm = torch.empty(1, dtype=torch.float32, device=ref.device)
    else:
        _match(norm, "norm", (1,), torch.float32, dev)
    if outs is None:
        outs = [torch.empty_like(g) for g in grads]
    elif len(outs) != n:
        raise ValueError("%d outputs for %d gradients" % (len(outs), n))
    elif list(map(tensor.numel, outs)) != sizes or [o.dtype for o in outs] != types \
            or any(map(dev.__ne__, map(tensor.get_device, outs))) \
            or not all(map(tensor.is_contiguous, outs)):
        for k in range(n):
            if outs[k].numel() != sizes[k]:
                raise ValueError("outs[%d] has %d elements, grads[%d] %d"
                                 % (k, outs[k].numel(), k, sizes[k]))
            _match(outs[k], "outs[%d]" % k, outs[k].shape, types[k], dev)
    pointers, L = ctypes.c_void_p * n, lib()
    ws = _scratch(L.ttt_clip_workspace_bytes(), ref, workspace)
    rc = L.ttt_clip_grad_norm(n, pointers(*map(tensor.data_ptr, grads)),
                              pointers(*map(tensor.data_ptr, outs)),
                              (ctypes.c_longlong * n)(*sizes),
                              (ctypes.c_int * n)(*kinds), max_norm, eps, norm.data_ptr(),
                              ws.data_ptr(), ws.numel(), _raw_stream(dev))
    if rc != OK:
        raise TTTError(rc, "ttt_clip_grad_norm")
    return outs, norm
