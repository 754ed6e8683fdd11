"""Thin Python front end of libpararnn (include/pararnn.h).

Argument marshalling only: torch tensors are passed as raw device pointers
with the current HIP stream; every step of the solve runs in the library's
kernels.  There is no fallback: if the library is missing or a call fails,
this module raises.
"""
from __future__ import annotations

import ctypes as C
import os
import struct

import numpy as np

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libpararnn.so")

# status codes (include/pararnn.h)
PR_OK, PR_EINVAL, PR_EWORKSPACE, PR_EHIP, PR_EUNSUPPORTED, PR_ELOOKBACK = 0, -1, -2, -3, -5, -6
PR_NOT_CONVERGED, PR_NONFINITE = 1, 2
PR_F32, PR_BF16 = 0, 1
PR_JAC_DENSE, PR_JAC_DIAG, PR_JAC_BLOCK2, PR_JAC_ZERO = 0, 1, 2, 3

EXPORTS = ["pararnn_workspace_bytes", "pararnn_solve", "pararnn_adjoint", "pararnn_solve_adjoint",
           "pararnn_scan_workspace_bytes", "pararnn_affine_scan", "pararnn_strerror", "pararnn_last_error", "pararnn_trace", "pararnn_trace_read",
           "pararnn_trace_kernel", "pararnn_lsim_workspace_bytes", "pararnn_lsim", "pararnn_elk_workspace_bytes",
           "pararnn_solve_elk", "pararnn_affine_scan_noalloc", "pararnn_conv", "pararnn_conv_workspace_bytes",
           "pararnn_conv_adjoint", "pararnn_conv_step", "pararnn_ssm_workspace_bytes", "pararnn_ssm_scan",
           "pararnn_ssm_adjoint", "pararnn_ssm_step", "pararnn_rmsnorm", "pararnn_rmsnorm_workspace_bytes",
           "pararnn_rmsnorm_adjoint", "pararnn_quant_rows", "pararnn_gemm_i8_workspace_bytes", "pararnn_gemm_i8",
           "pararnn_gated_workspace_bytes", "pararnn_gated_scan", "pararnn_gated_adjoint", "pararnn_gated_step",
           "pararnn_block_norm", "pararnn_block_norm_workspace_bytes", "pararnn_block_norm_adjoint", "pararnn_gemm_w4",
           "pararnn_quant_w4", "pararnn_dequant_w4"]
NOALLOC_SCRATCH_BYTES = 16 << 20  # PR_NOALLOC_SCRATCH_BYTES
SSM_STATE_STEPS = 16  # PR_SSM_STATE_STEPS
GATED_STATE_STEPS = 64  # PR_GATED_STATE_STEPS
GATES = {"silu": 1, "sigmoid": 2}  # PR_GATE_*


class Problem(C.Structure):
    _fields_ = [("cell", C.c_int), ("jac", C.c_int), ("dtype", C.c_int), ("B", C.c_int), ("T", C.c_int),
                ("d", C.c_int), ("n", C.c_int)]


class Weights(C.Structure):
    _fields_ = [("W_x", C.c_void_p), ("b_x", C.c_void_p), ("W_h", C.c_void_p), ("b_h", C.c_void_p),
                ("peep", C.c_void_p)]


class Grads(C.Structure):
    _fields_ = [("W_x", C.c_void_p), ("b_x", C.c_void_p), ("W_h", C.c_void_p), ("b_h", C.c_void_p),
                ("peep", C.c_void_p)]


class View(C.Structure):
    """pr_view: a [B, T, channels] array with adjacent channels."""
    _fields_ = [("p", C.c_void_p), ("sb", C.c_longlong), ("st", C.c_longlong)]


class Rows(C.Structure):
    _fields_ = [("p", C.c_void_p), ("ld", C.c_longlong)]


class ConvProblem(C.Structure):
    _fields_ = [("dtype", C.c_int), ("B", C.c_int), ("T", C.c_int), ("D", C.c_int), ("W", C.c_int), ("silu", C.c_int)]


class SsmProblem(C.Structure):
    _fields_ = [("dtype", C.c_int), ("B", C.c_int), ("T", C.c_int), ("D", C.c_int), ("N", C.c_int), ("G", C.c_int),
                ("softplus", C.c_int)]


class SsmInputs(C.Structure):
    _fields_ = [("u", View), ("dt", View), ("z", View), ("B", View), ("C", View), ("A", C.c_void_p),
                ("D", C.c_void_p), ("dt_bias", C.c_void_p), ("h0", C.c_void_p), ("lengths", C.c_void_p)]


class _SsmInputsFlat(C.Structure):
    """The same layout without nested structures, which take longer to fill."""
    _fields_ = [(a + "_" + f, c) for a in ("u", "dt", "z", "B", "C")
                for f, c in (("p", C.c_void_p), ("sb", C.c_longlong), ("st", C.c_longlong))] + [
        (a, C.c_void_p) for a in ("A", "D", "dt_bias", "h0", "lengths")]


class SsmGrads(C.Structure):
    _fields_ = [("u", View), ("dt", View), ("z", View), ("B", View), ("C", View), ("A", C.c_void_p),
                ("D", C.c_void_p), ("dt_bias", C.c_void_p), ("h0", C.c_void_p)]


class GatedProblem(C.Structure):
    _fields_ = [("dtype", C.c_int), ("B", C.c_int), ("T", C.c_int), ("D", C.c_int)]


class GatedInputs(C.Structure):
    _fields_ = [("x", View), ("r", View), ("i", View), ("decay", C.c_void_p), ("r_bias", C.c_void_p),
                ("i_bias", C.c_void_p), ("h0", C.c_void_p), ("lengths", C.c_void_p)]


class GatedGrads(C.Structure):
    _fields_ = [("x", View), ("r", View), ("i", View), ("decay", C.c_void_p), ("r_bias", C.c_void_p),
                ("i_bias", C.c_void_p), ("h0", C.c_void_p)]


class BlockNormProblem(C.Structure):
    _fields_ = [("dtype", C.c_int), ("n", C.c_int), ("rows", C.c_longlong), ("eps", C.c_float), ("gate", C.c_int)]


class BlockNormGrads(C.Structure):
    _fields_ = [("x", Rows), ("z", Rows), ("res", Rows), ("w", C.c_void_p), ("scale", C.c_void_p),
                ("w_next", C.c_void_p)]


class NormProblem(C.Structure):
    _fields_ = [("dtype", C.c_int), ("n", C.c_int), ("rows", C.c_longlong), ("eps", C.c_float)]


class PararnnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {strerror(status)} ({status}): {last_error()}")


_lib = None


def lib():
    """Load libpararnn.so (raises if it has not been built)."""
    global _lib, _several_gpus
    if _lib is None:
        import torch
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: run __graft_entry__.build() first")
        L = C.CDLL(LIB_PATH)
        P, I, F, S = C.c_void_p, C.c_int, C.c_float, C.c_size_t
        L.pararnn_workspace_bytes.argtypes = [P, I]
        L.pararnn_workspace_bytes.restype = S
        L.pararnn_solve.argtypes = [P, P, P, P, F, I, P, P, P, I, P, S, P]
        L.pararnn_solve.restype = I
        L.pararnn_adjoint.argtypes = [P, P, P, P, P, P, P, P, P, P, P, S, P]
        L.pararnn_adjoint.restype = I
        L.pararnn_solve_adjoint.argtypes = [P, P, P, P, F, I, P, P, P, I, P, P, P, P, P, P, S, P]
        L.pararnn_solve_adjoint.restype = I
        L.pararnn_scan_workspace_bytes.argtypes = [I, I, I, I]
        L.pararnn_scan_workspace_bytes.restype = S
        L.pararnn_affine_scan.argtypes = [I, I, I, I, I, P, P, P, P, S, P]
        L.pararnn_affine_scan.restype = I
        L.pararnn_affine_scan_noalloc.argtypes = [I, I, I, I, I, P, P, P, P]
        L.pararnn_affine_scan_noalloc.restype = I
        L.pararnn_strerror.argtypes = [I]
        L.pararnn_strerror.restype = C.c_char_p
        L.pararnn_last_error.argtypes = []
        L.pararnn_last_error.restype = C.c_char_p
        L.pararnn_trace.argtypes = [I]
        L.pararnn_trace.restype = I
        L.pararnn_trace_read.argtypes = [P, P, P, P]
        L.pararnn_trace_read.restype = I
        L.pararnn_trace_kernel.argtypes = [I, P, P]
        L.pararnn_trace_kernel.restype = I
        L.pararnn_lsim_workspace_bytes.argtypes = [I, I, I, I, I]
        L.pararnn_lsim_workspace_bytes.restype = S
        L.pararnn_lsim.argtypes = [I, I, I, I, I, P, P, P, P, F, P, P, P, P, P, S, P]
        L.pararnn_lsim.restype = I
        L.pararnn_elk_workspace_bytes.argtypes = [P]
        L.pararnn_elk_workspace_bytes.restype = S
        L.pararnn_solve_elk.argtypes = [P, P, P, P, F, F, I, P, P, P, I, P, S, P]
        L.pararnn_solve_elk.restype = I
        LL = C.c_longlong
        for name, res, args in (
                ("conv", I, [P, P, P, P, P, P, P, P, P]),
                ("conv_workspace_bytes", S, [P]),
                ("conv_adjoint", I, [P, P, P, P, P, P, P, P, P, P, P, P, P, S, P]),
                ("conv_step", I, [P, P, P, P, P, I, P, P, P]),
                ("ssm_workspace_bytes", S, [P, I]),
                ("ssm_scan", I, [P, P, P, P, P, P, S, P]),
                ("ssm_adjoint", I, [P, P, P, P, P, P, P, S, P]),
                ("ssm_step", I, [P, P, P, P, I, P, P]),
                ("rmsnorm", I, [P, P, P, P, P, P, P, P, P]),
                ("rmsnorm_workspace_bytes", S, [P]),
                ("rmsnorm_adjoint", I, [P, P, P, P, P, P, P, P, S, P]),
                ("quant_rows", I, [P, P, P, P, P]),
                ("gemm_i8_workspace_bytes", S, [I, I, I]),
                ("gemm_i8", I, [I, I, I, I, P, LL, P, P, LL, P, P, P, LL, P, S, P]),
                ("gated_workspace_bytes", S, [P, I]),
                ("gated_scan", I, [P, P, P, P, P, P, S, P]),
                ("gated_adjoint", I, [P, P, P, P, P, P, P, S, P]),
                ("gated_step", I, [P, P, P, P, I, P, P]),
                ("block_norm", I, [P, P, P, P, P, P, P, P, P, P]),
                ("block_norm_workspace_bytes", S, [P]),
                ("block_norm_adjoint", I, [P, P, P, P, P, P, P, P, P, P, P, S, P]),
                ("gemm_w4", I, [I, I, I, I, I, P, LL, P, LL, P, P, P, P, LL, P]),
                ("quant_w4", I, [I, I, I, I, P, LL, P, LL, P, P, P]),
                ("dequant_w4", I, [I, I, I, I, P, LL, P, P, P, LL, P])):
            f = getattr(L, "pararnn_" + name)
            f.restype, f.argtypes = res, args
        _several_gpus = torch.cuda.device_count() > 1
        _lib = L
    return _lib


def strerror(status: int) -> str:
    return lib().pararnn_strerror(status).decode()


def last_error() -> str:
    return lib().pararnn_last_error().decode()


def _p(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream():
    import torch
    return C.c_void_p(torch.cuda.current_stream().cuda_stream)


def make_problem(cell, jac, dtype, B, T, d, n) -> Problem:
    return Problem(cell, jac, dtype, B, T, d, n)


def make_weights(W_x, b_x, W_h, b_h, peep=None) -> Weights:
    return Weights(_p(W_x), _p(b_x), _p(W_h), _p(b_h), _p(peep))


def workspace_bytes(prob: Problem, with_adjoint: bool = True) -> int:
    return lib().pararnn_workspace_bytes(C.byref(prob), int(with_adjoint))


def solve(prob: Problem, w: Weights, x, h0, tol: float, max_iters: int, h, workspace, hist_cap: int = 64,
          check: bool = True):
    """Runs pararnn_solve; returns (status, iters, delta history)."""
    it = C.c_int(0)
    hist = np.zeros(max(hist_cap, 1), dtype=np.float32)
    st = lib().pararnn_solve(C.byref(prob), C.byref(w), _p(x), _p(h0), float(tol), int(max_iters), _p(h),
                             C.byref(it), hist.ctypes.data_as(C.c_void_p), int(hist_cap), _p(workspace),
                             workspace.numel() * workspace.element_size(), _stream())
    if check and st < 0:
        raise PararnnError(st, "pararnn_solve")
    return st, it.value, hist[:min(it.value, hist_cap)].copy()


def elk_workspace_bytes(prob: Problem) -> int:
    return lib().pararnn_elk_workspace_bytes(C.byref(prob))


def solve_elk(prob: Problem, w: Weights, x, h0, lam: float, tol: float, max_iters: int, h, workspace,
              hist_cap: int = 64, check: bool = True):
    """Runs pararnn_solve_elk (quasi-ELK, damping lam); returns (status, iters, delta history)."""
    it = C.c_int(0)
    hist = np.zeros(max(hist_cap, 1), dtype=np.float32)
    st = lib().pararnn_solve_elk(C.byref(prob), C.byref(w), _p(x), _p(h0), float(lam), float(tol), int(max_iters),
                                 _p(h), C.byref(it), hist.ctypes.data_as(C.c_void_p), int(hist_cap), _p(workspace),
                                 workspace.numel() * workspace.element_size(), _stream())
    if check and st < 0:
        raise PararnnError(st, "pararnn_solve_elk")
    return st, it.value, hist[:min(it.value, hist_cap)].copy()


def adjoint(prob: Problem, w: Weights, x, h0, h, g, workspace, lam=None, dx=None, dh0=None, grads: dict | None = None,
            check: bool = True) -> int:
    gr = None
    if grads is not None:
        gr = Grads(*[_p(grads.get(k)) for k in ("W_x", "b_x", "W_h", "b_h", "peep")])
    st = lib().pararnn_adjoint(C.byref(prob), C.byref(w), _p(x), _p(h0), _p(h), _p(g), _p(lam), _p(dx), _p(dh0),
                               C.byref(gr) if gr is not None else None, _p(workspace),
                               workspace.numel() * workspace.element_size(), _stream())
    if check and st < 0:
        raise PararnnError(st, "pararnn_adjoint")
    return st


def solve_adjoint(prob: Problem, w: Weights, x, h0, tol: float, max_iters: int, h, g, workspace, lam=None, dx=None,
                  dh0=None, grads: dict | None = None, hist_cap: int = 64, check: bool = True):
    """Runs pararnn_solve_adjoint; returns (status, iters, delta history)."""
    it = C.c_int(0)
    hist = np.zeros(max(hist_cap, 1), dtype=np.float32)
    gr = None
    if grads is not None:
        gr = Grads(*[_p(grads.get(k)) for k in ("W_x", "b_x", "W_h", "b_h", "peep")])
    st = lib().pararnn_solve_adjoint(C.byref(prob), C.byref(w), _p(x), _p(h0), float(tol), int(max_iters), _p(h),
                                     C.byref(it), hist.ctypes.data_as(C.c_void_p), int(hist_cap), _p(g), _p(lam),
                                     _p(dx), _p(dh0), C.byref(gr) if gr is not None else None, _p(workspace),
                                     workspace.numel() * workspace.element_size(), _stream())
    if check and st < 0:
        raise PararnnError(st, "pararnn_solve_adjoint")
    return st, it.value, hist[:min(it.value, hist_cap)].copy()


def trace(enable: bool) -> None:
    st = lib().pararnn_trace(int(enable))
    if st < 0:
        raise PararnnError(st, "pararnn_trace")


def trace_read() -> dict:
    sm, sl, am, al = C.c_double(0), C.c_longlong(0), C.c_double(0), C.c_longlong(0)
    st = lib().pararnn_trace_read(C.byref(sm), C.byref(sl), C.byref(am), C.byref(al))
    if st < 0:
        raise PararnnError(st, "pararnn_trace_read")
    return dict(sweep_ms=sm.value, sweep_launches=sl.value, adjoint_ms=am.value, adjoint_launches=al.value)


TRACE_SWEEP, TRACE_ADJOINT, TRACE_PROJECTION, TRACE_ADJOINT_PRODUCTS, TRACE_DENSE_PRODUCTS = 0, 1, 2, 3, 4
TRACE_LSIM = 5


def trace_kernel(which: int):
    """(total ms, launches) of one traced category."""
    ms, n = C.c_double(0), C.c_longlong(0)
    st = lib().pararnn_trace_kernel(int(which), C.byref(ms), C.byref(n))
    if st < 0:
        raise PararnnError(st, "pararnn_trace_kernel")
    return ms.value, n.value


def scan_workspace_bytes(jac: int, B: int, T: int, n: int) -> int:
    return lib().pararnn_scan_workspace_bytes(jac, B, T, n)


def affine_scan(jac: int, A, b, y, workspace, reverse: bool = False, check: bool = True) -> int:
    B, T, n = b.shape[0], b.shape[1], b.shape[2]
    st = lib().pararnn_affine_scan(jac, B, T, n, int(reverse), _p(A), _p(b), _p(y), _p(workspace),
                                   workspace.numel() * workspace.element_size(), _stream())
    if check and st < 0:
        raise PararnnError(st, "pararnn_affine_scan")
    return st


def affine_scan_noalloc(jac: int, A, b, y, reverse: bool = False, check: bool = True) -> int:
    """pararnn_affine_scan_noalloc: the same scan with the library's static
    device scratch instead of a workspace."""
    B, T, n = b.shape[0], b.shape[1], b.shape[2]
    st = lib().pararnn_affine_scan_noalloc(jac, B, T, n, int(reverse), _p(A), _p(b), _p(y), _stream())
    if check and st < 0:
        raise PararnnError(st, "pararnn_affine_scan_noalloc")
    return st


def lsim_workspace_bytes(B: int, T: int, nx: int, m: int, p: int) -> int:
    return lib().pararnn_lsim_workspace_bytes(B, T, nx, m, p)


def lsim(A, Bm, Cm, Dm, dt: float, U, x0, x, y, workspace, check: bool = True) -> int:
    """pararnn_lsim on fp32 device tensors: U [B,T,m], x0 [B,nx] or None,
    outputs x [B,T,nx] (or None) and y [B,T,p]."""
    import torch
    for name, t in (("A", A), ("B", Bm), ("C", Cm), ("D", Dm), ("U", U), ("x0", x0), ("x", x), ("y", y)):
        if t is not None and (t.dtype != torch.float32 or not t.is_contiguous()):
            raise ValueError(f"lsim: {name} must be a contiguous float32 tensor, got {t.dtype}")
    B, T, m = U.shape[0], U.shape[1], U.shape[2]
    nx, p = A.shape[0], Cm.shape[0]
    st = lib().pararnn_lsim(B, T, nx, m, p, _p(A), _p(Bm), _p(Cm), _p(Dm), float(dt), _p(U), _p(x0), _p(x), _p(y),
                            _p(workspace), workspace.numel() * workspace.element_size(), _stream())
    if check and st < 0:
        raise PararnnError(st, "pararnn_lsim")
    return st


# ---------------------------------------------------------------------------
# operators of a selective state space block
# ---------------------------------------------------------------------------
def _dtype_code(dt, what):
    import torch
    if dt == torch.bfloat16:
        return PR_BF16
    if dt == torch.float32:
        return PR_F32
    raise ValueError(f"{what}: storage must be float32 or bfloat16, got {dt}")


def _strides(where, name, t, shape, adjacent):
    step = 1
    for k in range(1, adjacent + 1):
        if shape[-k] != 1 and t.stride(-k) != step:
            raise ValueError(f"{where}: the last {adjacent} axes of {name} must be contiguous, got strides {t.stride()}")
        step *= shape[-k]


_several_gpus = False  # set where the library is loaded


def _same_device(where, name, t):
    """Kernels are launched on the current device, for its memory and its stream."""
    import torch
    if t.get_device() != torch.cuda.current_device():
        raise ValueError(f"{where}: {name} is on GPU {t.get_device()}, the current one is {torch.cuda.current_device()}")


# These checks run on every call, single tokens' included, so they take the
# short way through torch's attributes first.
def _need(where, name, t, shape, dtype):
    """The address of tensor t after a check of its shape, type, device and
    adjacent last axis."""
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{where}: {name} must be a {dtype} tensor of shape {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{where}: {name} must be on the GPU")
    if _several_gpus:
        _same_device(where, name, t)
    if t.stride(-1) != 1:
        _strides(where, name, t, shape, 1)
    return t.data_ptr()


def _dense(where, name, t, shape, dtype):
    """The address of t, all of whose axes must be contiguous; None passes."""
    if t is None:
        return None
    if t.dtype != dtype or t.shape != shape or not t.is_cuda or _several_gpus or not t.is_contiguous():
        _need(where, name, t, shape, dtype)
        _strides(where, name, t, shape, len(shape))
    return t.data_ptr()


def _flat(where, name, t, shape, dtype):
    """The fields of a pr_view of t [B, T, channels] or, for single tokens, [B, channels]."""
    if t is None:
        return None, 0, 0
    p = _need(where, name, t, shape, dtype)
    s = t.stride()
    return (p, s[0], s[1]) if len(s) == 3 else (p, s[0], 0)


def _view(where, name, t, shape, dtype):
    return View(*_flat(where, name, t, shape, dtype))


def _stream_of(t):
    """The raw handle of the current stream of t's device, which is the current one."""
    import torch
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _rows(where, name, t, shape, dtype):
    if t is None:
        return None
    return C.byref(Rows(_need(where, name, t, shape, dtype), t.stride(0)))  # (one row: any stride)


def _done(st, where, check=True):
    if check and st < 0:
        raise PararnnError(st, where)
    return st


def _ws(where, workspace):
    """Address and bytes of the workspace, into which kernels write."""
    if not workspace.is_contiguous():
        raise ValueError(f"{where}: the workspace must be contiguous, got strides {workspace.stride()}")
    if not workspace.is_cuda:
        raise ValueError(f"{where}: the workspace must be on the GPU")
    if _several_gpus:
        _same_device(where, "the workspace", workspace)
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def conv_workspace_bytes(dtype, B: int, T: int, D: int, W: int) -> int:
    """Workspace of conv_adjoint for sequences stored in the torch type dtype."""
    return lib().pararnn_conv_workspace_bytes(C.byref(ConvProblem(_dtype_code(dtype, "conv"), B, T, D, W, 1)))


def conv(x, w, bias, y, state_in=None, state_out=None, lengths=None, silu: bool = True, check: bool = True) -> int:
    """pararnn_conv: short causal convolution of x [B, T, D] with w [D, W] into y."""
    import torch
    (B, T, D), W, dt, n = x.shape, w.shape[1], x.dtype, "conv"
    pb = ConvProblem(_dtype_code(dt, n), B, T, D, W, int(silu))
    st = lib().pararnn_conv(C.byref(pb), C.byref(_view(n, "x", x, (B, T, D), dt)), _dense(n, "w", w, (D, W), dt),
                            _dense(n, "bias", bias, (D,), dt), _dense(n, "state_in", state_in, (B, W - 1, D), dt),
                            _dense(n, "lengths", lengths, (B,), torch.int32),
                            C.byref(_view(n, "y", y, (B, T, D), dt)),
                            _dense(n, "state_out", state_out, (B, W - 1, D), dt), _stream_of(x))
    return _done(st, "pararnn_conv", check)


def conv_adjoint(x, w, bias, dy, dx, dw, dbias, workspace, state_in=None, dstate_out=None, dstate_in=None, lengths=None,
                 silu: bool = True, check: bool = True) -> int:
    """pararnn_conv_adjoint: gradients of conv; dx, dw, dbias and dstate_in may be None."""
    import torch
    (B, T, D), W, dt, n, f32 = x.shape, w.shape[1], x.dtype, "conv_adjoint", torch.float32
    pb = ConvProblem(_dtype_code(dt, n), B, T, D, W, int(silu))
    st = lib().pararnn_conv_adjoint(
        C.byref(pb), C.byref(_view(n, "x", x, (B, T, D), dt)), _dense(n, "w", w, (D, W), dt),
        _dense(n, "bias", bias, (D,), dt), _dense(n, "state_in", state_in, (B, W - 1, D), dt),
        _dense(n, "lengths", lengths, (B,), torch.int32), C.byref(_view(n, "dy", dy, (B, T, D), dt)),
        _dense(n, "dstate_out", dstate_out, (B, W - 1, D), dt), C.byref(_view(n, "dx", dx, (B, T, D), dt)),
        _dense(n, "dw", dw, (D, W), f32), _dense(n, "dbias", dbias, (D,), f32),
        _dense(n, "dstate_in", dstate_in, (B, W - 1, D), dt), *_ws(n, workspace), _stream_of(x))
    return _done(st, "pararnn_conv_adjoint", check)


def conv_step(x, w, bias, state, y, slots=None, silu: bool = True, check: bool = True) -> int:
    """pararnn_conv_step: one token x [B, D] per sequence on the pool state [slots, W - 1, D]."""
    import torch
    (B, D), W, dt, n = x.shape, w.shape[1], x.dtype, "conv_step"
    pb = ConvProblem(_dtype_code(dt, n), B, 1, D, W, int(silu))
    pool = state.shape[0]
    st = lib().pararnn_conv_step(C.byref(pb), C.byref(_view(n, "x", x, (B, D), dt)), _dense(n, "w", w, (D, W), dt),
                                 _dense(n, "bias", bias, (D,), dt), _dense(n, "state", state, (pool, W - 1, D), dt),
                                 pool, _dense(n, "slots", slots, (B,), torch.int32),
                                 C.byref(_view(n, "y", y, (B, D), dt)), _stream_of(x))
    return _done(st, "pararnn_conv_step", check)


def ssm_workspace_bytes(dtype, B: int, T: int, D: int, N: int, G: int = 1, with_adjoint: bool = True) -> int:
    pb = SsmProblem(_dtype_code(dtype, "ssm"), B, T, D, N, G, 1)
    return lib().pararnn_ssm_workspace_bytes(C.byref(pb), int(with_adjoint))


def ssm_states_shape(B: int, T: int, D: int, N: int):
    """Shape of the fp32 states that ssm_scan saves for ssm_scan_adjoint."""
    return B, -(-T // SSM_STATE_STEPS), D, N


def _ssm(where, axes, u, dt, A, Bm, Cm, D, z, dt_bias, h0, lengths, softplus):
    import torch
    lib()  # before the tensors' checks, which depend on the GPUs there are
    st, f32 = u.dtype, torch.float32
    shape, (ch, N) = u.shape, A.shape
    if len(shape) != axes:
        raise ValueError(f"{where}: u must be [B, {'T, ' if axes == 3 else ''}channels], got {tuple(shape)}")
    B, T = shape[0], shape[1] if axes == 3 else 1
    width = Bm.shape[-1]
    if width % N or not width:
        raise ValueError(f"{where}: B has {width} columns, not a multiple of the {N} states of A")
    bc = shape[:-1] + (width,)
    pb = SsmProblem(_dtype_code(st, where), B, T, shape[-1], N, width // N, int(softplus))
    return pb, _SsmInputsFlat(
        *_flat(where, "u", u, shape, st), *_flat(where, "dt", dt, shape, st), *_flat(where, "z", z, shape, st),
        *_flat(where, "B", Bm, bc, st), *_flat(where, "C", Cm, bc, st), _dense(where, "A", A, (shape[-1], N), f32),
        _dense(where, "D", D, (ch,), f32), _dense(where, "dt_bias", dt_bias, (ch,), f32),
        _dense(where, "h0", h0, (B, ch, N), f32), _dense(where, "lengths", lengths, (B,), torch.int32))


def ssm_scan(u, dt, A, Bm, Cm, y, workspace, D=None, z=None, dt_bias=None, h0=None, h_last=None, states=None,
             lengths=None, softplus: bool = True, check: bool = True) -> int:
    """pararnn_ssm_scan: the selective scan of u [B, T, channels] into y."""
    import torch
    n = "ssm_scan"
    pb, inp = _ssm(n, 3, u, dt, A, Bm, Cm, D, z, dt_bias, h0, lengths, softplus)
    st = lib().pararnn_ssm_scan(
        C.byref(pb), C.byref(inp), C.byref(_view(n, "y", y, u.shape, u.dtype)),
        _dense(n, "h_last", h_last, (pb.B, pb.D, pb.N), torch.float32),
        _dense(n, "states", states, ssm_states_shape(pb.B, pb.T, pb.D, pb.N), torch.float32), *_ws(n, workspace),
        _stream_of(u))
    return _done(st, "pararnn_ssm_scan", check)


def ssm_scan_adjoint(u, dt, A, Bm, Cm, states, dy, workspace, D=None, z=None, dt_bias=None, lengths=None, dh_last=None,
                     du=None, ddt=None, dz=None, dB=None, dC=None, dA=None, dD=None, ddt_bias=None, dh0=None,
                     softplus: bool = True, check: bool = True) -> int:
    """pararnn_ssm_adjoint: gradients of ssm_scan from the states it saved; any output may be None."""
    import torch
    n, f32 = "ssm_scan_adjoint", torch.float32
    pb, inp = _ssm(n, 3, u, dt, A, Bm, Cm, D, z, dt_bias, None, lengths, softplus)
    shape, bc, t = u.shape, Bm.shape, u.dtype
    gr = SsmGrads(_view(n, "du", du, shape, t), _view(n, "ddt", ddt, shape, t), _view(n, "dz", dz, shape, t),
                  _view(n, "dB", dB, bc, t), _view(n, "dC", dC, bc, t), _dense(n, "dA", dA, (pb.D, pb.N), f32),
                  _dense(n, "dD", dD, (pb.D,), f32), _dense(n, "ddt_bias", ddt_bias, (pb.D,), f32),
                  _dense(n, "dh0", dh0, (pb.B, pb.D, pb.N), f32))
    st = lib().pararnn_ssm_adjoint(
        C.byref(pb), C.byref(inp), _dense(n, "states", states, ssm_states_shape(pb.B, pb.T, pb.D, pb.N), f32),
        C.byref(_view(n, "dy", dy, shape, t)), _dense(n, "dh_last", dh_last, (pb.B, pb.D, pb.N), f32), C.byref(gr),
        *_ws(n, workspace), _stream_of(u))
    return _done(st, "pararnn_ssm_adjoint", check)


def ssm_step(u, dt, A, Bm, Cm, state, y, D=None, z=None, dt_bias=None, slots=None, softplus: bool = True,
             check: bool = True) -> int:
    """pararnn_ssm_step: one token u [B, channels] per sequence on the fp32 pool state [slots, channels, N]."""
    import torch
    n = "ssm_step"
    pb, inp = _ssm(n, 2, u, dt, A, Bm, Cm, D, z, dt_bias, None, None, softplus)
    pool = state.shape[0]
    st = lib().pararnn_ssm_step(C.byref(pb), C.byref(inp), C.byref(_view(n, "y", y, u.shape, u.dtype)),
                                _dense(n, "state", state, (pool, pb.D, pb.N), torch.float32), pool,
                                _dense(n, "slots", slots, (pb.B,), torch.int32), _stream_of(u))
    return _done(st, "pararnn_ssm_step", check)


def rmsnorm(x, w, y=None, residual=None, sum_out=None, q=None, scale=None, eps: float = 1e-5,
            check: bool = True) -> int:
    """pararnn_rmsnorm of x [rows, n] (+ residual): y, or q (int8) with scale [rows]."""
    import torch
    (rows, n), dt, where = x.shape, x.dtype, "rmsnorm"
    pb = NormProblem(_dtype_code(dt, where), n, rows, eps)
    st = lib().pararnn_rmsnorm(
        C.byref(pb), _rows(where, "x", x, (rows, n), dt), _rows(where, "residual", residual, (rows, n), dt),
        _dense(where, "w", w, (n,), dt), _rows(where, "sum_out", sum_out, (rows, n), dt),
        _rows(where, "y", y, (rows, n), dt), _rows(where, "q", q, (rows, n), torch.int8),
        _dense(where, "scale", scale, (rows,), torch.float32), _stream_of(x))
    return _done(st, "pararnn_rmsnorm", check)


def rmsnorm_workspace_bytes(dtype, rows: int, n: int) -> int:
    return lib().pararnn_rmsnorm_workspace_bytes(C.byref(NormProblem(_dtype_code(dtype, "rmsnorm"), n, rows, 0.0)))


def rmsnorm_adjoint(s, w, dy, dx, dw, workspace, dsum=None, eps: float = 1e-5, check: bool = True) -> int:
    """pararnn_rmsnorm_adjoint at the stored sum s [rows, n]; dx and dw may be None."""
    import torch
    (rows, n), dt, where = s.shape, s.dtype, "rmsnorm_adjoint"
    pb = NormProblem(_dtype_code(dt, where), n, rows, eps)
    st = lib().pararnn_rmsnorm_adjoint(
        C.byref(pb), _rows(where, "s", s, (rows, n), dt), _dense(where, "w", w, (n,), dt),
        _rows(where, "dy", dy, (rows, n), dt), _rows(where, "dsum", dsum, (rows, n), dt),
        _rows(where, "dx", dx, (rows, n), dt), _dense(where, "dw", dw, (n,), torch.float32), *_ws(where, workspace), _stream_of(s))
    return _done(st, "pararnn_rmsnorm_adjoint", check)


def quant_rows(x, q, scale, check: bool = True) -> int:
    """pararnn_quant_rows: x [rows, n] in 8 bits, q int8 and scale [rows]."""
    import torch
    (rows, n), dt, where = x.shape, x.dtype, "quant_rows"
    pb = NormProblem(_dtype_code(dt, where), n, rows, 0.0)
    st = lib().pararnn_quant_rows(C.byref(pb), _rows(where, "x", x, (rows, n), dt),
                                  _rows(where, "q", q, (rows, n), torch.int8),
                                  _dense(where, "scale", scale, (rows,), torch.float32), _stream_of(x))
    return _done(st, "pararnn_quant_rows", check)


def gemm_i8_workspace_bytes(M: int, N: int, K: int) -> int:
    return lib().pararnn_gemm_i8_workspace_bytes(M, N, K)


def gemm_i8(a, a_scale, w, w_scale, out, workspace, bias=None, check: bool = True) -> int:
    """pararnn_gemm_i8: out [M, N] = (a w^T) a_scale w_scale + bias for int8 a [M, K] and w [N, K]."""
    import torch
    (M, K), N, dt, n, f32 = a.shape, w.shape[0], out.dtype, "gemm_i8", torch.float32
    st = lib().pararnn_gemm_i8(
        _dtype_code(dt, n), M, N, K, _need(n, "a", a, (M, K), torch.int8), a.stride(0),
        _dense(n, "a_scale", a_scale, (M,), f32), _need(n, "w", w, (N, K), torch.int8), w.stride(0),
        _dense(n, "w_scale", w_scale, (N,), f32), _dense(n, "bias", bias, (N,), dt),
        _need(n, "out", out, (M, N), dt), out.stride(0), *_ws(n, workspace), _stream_of(a))
    return _done(st, "pararnn_gemm_i8", check)


# ---------------------------------------------------------------------------
# operators of a gated recurrent block
# ---------------------------------------------------------------------------
# Their structures are packed as bytes, in the C layout: single tokens' calls are
# bound by the work done here, and a ctypes structure takes several times as long.
_PACK_VIEW, _PACK_ROWS = struct.Struct("qqq").pack, struct.Struct("qq").pack
_PACK_GATED, _PACK_GATED_IN = struct.Struct("iiii").pack, struct.Struct("14q").pack
_PACK_GATED_GRADS, _PACK_BLOCK_NORM = struct.Struct("13q").pack, struct.Struct("iiqfi").pack
_PACK_BLOCK_NORM_GRADS = struct.Struct("9q").pack


def _strided(where, name, t, shape, dtype):
    """The address and the strides of t, whose last axis must be adjacent."""
    if t.dtype is not dtype or t.shape != shape or not t.is_cuda or _several_gpus:
        _need(where, name, t, shape, dtype)
    s = t.stride()
    if s[-1] != 1:
        _strides(where, name, t, shape, 1)
    return t.data_ptr(), s


def _address(where, name, t, shape, dtype):
    """The address of t, all of whose axes must be contiguous; 0 for None."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.shape != shape or not t.is_cuda or _several_gpus or not t.is_contiguous():
        return _dense(where, name, t, shape, dtype)
    return t.data_ptr()


def _seq(where, name, t, shape, dtype):
    """The fields of a pr_view of t [B, T, channels] or, for single tokens, [B, channels]."""
    if t is None:
        return 0, 0, 0
    p, s = _strided(where, name, t, shape, dtype)
    return p, s[0], s[1] if len(s) == 3 else 0


def _row2(where, name, t, shape, dtype):
    """The fields of a pr_rows of t."""
    if t is None:
        return 0, 0
    p, s = _strided(where, name, t, shape, dtype)
    return p, s[0]


def gated_workspace_bytes(dtype, B: int, T: int, D: int, with_adjoint: bool = True) -> int:
    return lib().pararnn_gated_workspace_bytes(_PACK_GATED(_dtype_code(dtype, "gated"), B, T, D), int(with_adjoint))


def gated_states_shape(B: int, T: int, D: int):
    """Shape of the fp32 states that gated_scan saves for gated_scan_adjoint."""
    return B, -(-T // GATED_STATE_STEPS), D


def _gated(where, axes, x, r, i, decay, r_bias, i_bias, h0, lengths):
    import torch
    lib()  # before the tensors' checks, which depend on the GPUs there are
    st, f32, shape = x.dtype, torch.float32, x.shape
    if len(shape) != axes:
        raise ValueError(f"{where}: x must be [B, {'T, ' if axes == 3 else ''}channels], got {tuple(shape)}")
    B, D = shape[0], shape[-1]
    ch = (D,)
    return shape, st, _PACK_GATED(_dtype_code(st, where), B, shape[1] if axes == 3 else 1, D), _PACK_GATED_IN(
        *_seq(where, "x", x, shape, st), *_seq(where, "r", r, shape, st), *_seq(where, "i", i, shape, st),
        _address(where, "decay", decay, ch, f32), _address(where, "r_bias", r_bias, ch, f32),
        _address(where, "i_bias", i_bias, ch, f32), _address(where, "h0", h0, (B, D), f32),
        _address(where, "lengths", lengths, (B,), torch.int32))


def gated_scan(x, r, i, decay, y, workspace, r_bias=None, i_bias=None, h0=None, h_last=None, states=None, lengths=None,
               check: bool = True) -> int:
    """pararnn_gated_scan: the gated recurrence of x [B, T, channels] with gates r and i into y."""
    import torch
    n, f32 = "gated_scan", torch.float32
    shape, t, pb, inp = _gated(n, 3, x, r, i, decay, r_bias, i_bias, h0, lengths)
    B, T, D = shape
    st = lib().pararnn_gated_scan(
        pb, inp, _PACK_VIEW(*_seq(n, "y", y, shape, t)), _address(n, "h_last", h_last, (B, D), f32),
        _address(n, "states", states, gated_states_shape(B, T, D), f32), *_ws(n, workspace), _stream_of(x))
    return _done(st, "pararnn_gated_scan", check)


def gated_scan_adjoint(x, r, i, decay, states, dy, workspace, r_bias=None, i_bias=None, lengths=None, dh_last=None,
                       dx=None, dr=None, di=None, ddecay=None, dr_bias=None, di_bias=None, dh0=None,
                       check: bool = True) -> int:
    """pararnn_gated_adjoint: gradients of gated_scan from the states it saved; any output may be None."""
    import torch
    n, f32 = "gated_scan_adjoint", torch.float32
    shape, t, pb, inp = _gated(n, 3, x, r, i, decay, r_bias, i_bias, None, lengths)
    B, T, D = shape
    ch = (D,)
    gr = _PACK_GATED_GRADS(
        *_seq(n, "dx", dx, shape, t), *_seq(n, "dr", dr, shape, t), *_seq(n, "di", di, shape, t),
        _address(n, "ddecay", ddecay, ch, f32), _address(n, "dr_bias", dr_bias, ch, f32),
        _address(n, "di_bias", di_bias, ch, f32), _address(n, "dh0", dh0, (B, D), f32))
    st = lib().pararnn_gated_adjoint(
        pb, inp, _address(n, "states", states, gated_states_shape(B, T, D), f32),
        _PACK_VIEW(*_seq(n, "dy", dy, shape, t)), _address(n, "dh_last", dh_last, (B, D), f32), gr,
        *_ws(n, workspace), _stream_of(x))
    return _done(st, "pararnn_gated_adjoint", check)


def gated_step(x, r, i, decay, state, y, r_bias=None, i_bias=None, slots=None, check: bool = True) -> int:
    """pararnn_gated_step: one token x [B, channels] per sequence on the fp32 pool state [slots, channels]."""
    import torch
    n = "gated_step"
    shape, t, pb, inp = _gated(n, 2, x, r, i, decay, r_bias, i_bias, None, None)
    pool = state.shape[0]
    st = lib().pararnn_gated_step(pb, inp, _PACK_VIEW(*_seq(n, "y", y, shape, t)),
                                  _address(n, "state", state, (pool, shape[1]), torch.float32), pool,
                                  _address(n, "slots", slots, (shape[0],), torch.int32), _stream_of(x))
    return _done(st, "pararnn_gated_step", check)


def _block_norm(where, x, z, gate, eps):
    """The shape and type of the rows x and the packed problem."""
    lib()
    shape, dt = x.shape, x.dtype
    if len(shape) != 2:
        raise ValueError(f"{where}: x must be [rows, n], got {tuple(shape)}")
    if gate not in GATES:
        raise ValueError(f"{where}: gate must be one of {sorted(GATES)}, got {gate!r}")
    return shape, dt, _PACK_BLOCK_NORM(_dtype_code(dt, where), shape[1], shape[0], eps, GATES[gate] if z is not None else 0)


def block_norm(x, w, t, z=None, gate: str = "silu", scale=None, residual=None, y=None, w_next=None, eps: float = 1e-5,
               check: bool = True) -> int:
    """pararnn_block_norm of x [rows, n]: t = residual + norm(x) w scale act(z) and, where y is given, y = norm(t) w_next."""
    n = "block_norm"
    shape, dt, pb = _block_norm(n, x, z, gate, eps)
    ch = (shape[1],)
    st = lib().pararnn_block_norm(
        pb, _PACK_ROWS(*_row2(n, "x", x, shape, dt)), None if z is None else _PACK_ROWS(*_row2(n, "z", z, shape, dt)),
        None if residual is None else _PACK_ROWS(*_row2(n, "residual", residual, shape, dt)),
        _address(n, "w", w, ch, dt), _address(n, "scale", scale, ch, dt), _address(n, "w_next", w_next, ch, dt),
        _PACK_ROWS(*_row2(n, "t", t, shape, dt)), None if y is None else _PACK_ROWS(*_row2(n, "y", y, shape, dt)),
        _stream_of(x))
    return _done(st, "pararnn_block_norm", check)


def block_norm_workspace_bytes(dtype, rows: int, n: int) -> int:
    """Workspace of block_norm_adjoint for rows stored in the torch type dtype."""
    return lib().pararnn_block_norm_workspace_bytes(_PACK_BLOCK_NORM(_dtype_code(dtype, "block_norm"), n, rows, 0.0, 0))


def block_norm_adjoint(x, w, dx, workspace, z=None, gate: str = "silu", scale=None, w_next=None, t=None, dt=None,
                       dy=None, dz=None, dres=None, dw=None, dscale=None, dw_next=None, eps: float = 1e-5,
                       check: bool = True) -> int:
    """pararnn_block_norm_adjoint: gradients of block_norm at x, z and the stored t from dt and dy; any output may be None."""
    import torch
    n, f32 = "block_norm_adjoint", torch.float32
    shape, st, pb = _block_norm(n, x, z, gate, eps)
    ch = (shape[1],)
    gr = _PACK_BLOCK_NORM_GRADS(*_row2(n, "dx", dx, shape, st), *_row2(n, "dz", dz, shape, st),
                                *_row2(n, "dres", dres, shape, st), _address(n, "dw", dw, ch, f32),
                                _address(n, "dscale", dscale, ch, f32), _address(n, "dw_next", dw_next, ch, f32))
    rc = lib().pararnn_block_norm_adjoint(
        pb, _PACK_ROWS(*_row2(n, "x", x, shape, st)), _PACK_ROWS(*_row2(n, "z", z, shape, st)),
        _address(n, "w", w, ch, st), _address(n, "scale", scale, ch, st), _address(n, "w_next", w_next, ch, st),
        _PACK_ROWS(*_row2(n, "t", t, shape, st)), _PACK_ROWS(*_row2(n, "dt", dt, shape, st)),
        _PACK_ROWS(*_row2(n, "dy", dy, shape, st)), gr, *_ws(n, workspace), _stream_of(x))
    return _done(rc, "pararnn_block_norm_adjoint", check)


def _w4(where, q, scale, zero, N, K, group, dt):
    """Addresses of a 4-bit weight matrix's parts: q, its row stride, scale, zero."""
    import torch
    if group < 1:
        raise ValueError(f"{where}: groups must have at least one column, got {group}")
    shape = (N, -(-K // group))
    return (*_row2(where, "q", q, (N, (K + 1) // 2), torch.uint8), _address(where, "scale", scale, shape, dt),
            _address(where, "zero", zero, shape, dt))


def gemm_w4(x, q, scale, out, group: int, zero=None, bias=None, check: bool = True) -> int:
    """pararnn_gemm_w4: out [M, N] = x [M, K] times the 4-bit weights q [N, (K + 1) / 2], plus bias."""
    n, dt = "gemm_w4", x.dtype
    lib()
    (M, K), N = x.shape, q.shape[0]
    st = lib().pararnn_gemm_w4(_dtype_code(dt, n), M, N, K, group, *_row2(n, "x", x, (M, K), dt),
                               *_w4(n, q, scale, zero, N, K, group, dt), _address(n, "bias", bias, (N,), dt),
                               *_row2(n, "out", out, (M, N), dt), _stream_of(x))
    return _done(st, "pararnn_gemm_w4", check)


def quant_w4(w, q, scale, group: int, zero=None, check: bool = True) -> int:
    """pararnn_quant_w4: w [N, K] in 4 bits, q uint8 [N, (K + 1) / 2] with scale (and zero) [N, groups]."""
    n, dt = "quant_w4", w.dtype
    lib()
    N, K = w.shape
    st = lib().pararnn_quant_w4(_dtype_code(dt, n), N, K, group, *_row2(n, "w", w, (N, K), dt),
                                *_w4(n, q, scale, zero, N, K, group, dt), _stream_of(w))
    return _done(st, "pararnn_quant_w4", check)


def dequant_w4(q, scale, w, group: int, zero=None, check: bool = True) -> int:
    """pararnn_dequant_w4: the values w [N, K] that q stands for."""
    n, dt = "dequant_w4", w.dtype
    lib()
    N, K = w.shape
    st = lib().pararnn_dequant_w4(_dtype_code(dt, n), N, K, group, *_w4(n, q, scale, zero, N, K, group, dt),
                                  *_row2(n, "w", w, (N, K), dt), _stream_of(w))
    return _done(st, "pararnn_dequant_w4", check)


# ---------------------------------------------------------------------------
# moving a problem (as drawn by synthetic.py) to the device
# ---------------------------------------------------------------------------
class DeviceProblem:
    """Device copies of a synthetic problem in its storage dtype, plus a workspace."""

    def __init__(self, p: dict, device="cuda", with_adjoint: bool = True, elk: bool = False):
        import torch
        from . import synthetic as sy
        self.p = p
        self.device = device
        self.prob = make_problem(p["cell"], p["jac"], p["dtype"], p["B"], p["T"], p["d"], p["n"])
        self.tdtype = torch.bfloat16 if p["dtype"] == PR_BF16 else torch.float32

        def up(a):
            if a is None:
                return None
            st = sy.to_storage(np.asarray(a), p["dtype"])
            if p["dtype"] == PR_BF16:
                return torch.from_numpy(st.view(np.int16).copy()).to(device).view(torch.bfloat16)
            return torch.from_numpy(st.copy()).to(device)

        self.W_x, self.b_x, self.W_h, self.b_h = up(p["W_x"]), up(p["b_x"]), up(p["W_h"]), up(p["b_h"])
        self.peep = up(p["peep"])
        self.x = up(p["x"])
        self.h0 = up(p["h0"])
        self.g = up(p["g"]) if p.get("g") is not None else None
        self.w = make_weights(self.W_x, self.b_x, self.W_h, self.b_h, self.peep)
        nbytes = workspace_bytes(self.prob, with_adjoint)
        if nbytes == 0:
            raise RuntimeError(f"pararnn_workspace_bytes: {last_error()}")
        if elk:
            nbytes = elk_workspace_bytes(self.prob)
            if nbytes == 0:
                raise RuntimeError(f"pararnn_elk_workspace_bytes: {last_error()}")
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.h = torch.empty((p["B"], p["T"], p["S"]), dtype=self.tdtype, device=device)

    def solve(self, tol=None, max_iters=None, hist_cap=64, check=True):
        p = self.p
        tol = p["tol"] if tol is None else tol
        max_iters = p["max_iters"] if max_iters is None else max_iters
        return solve(self.prob, self.w, self.x, self.h0, tol, max_iters, self.h, self.ws, hist_cap, check)

    def solve_elk(self, lam, tol=None, max_iters=None, hist_cap=64, check=True):
        p = self.p
        tol = p["tol"] if tol is None else tol
        max_iters = p["max_iters"] if max_iters is None else max_iters
        return solve_elk(self.prob, self.w, self.x, self.h0, lam, tol, max_iters, self.h, self.ws, hist_cap, check)

    def adjoint(self, h=None, g=None, want_grads=True, check=True):
        import torch
        p = self.p
        h = self.h if h is None else h
        g = self.g if g is None else g
        lam = torch.empty_like(h)
        dx = torch.empty_like(self.x)
        dh0 = torch.empty((p["B"], p["S"]), dtype=self.tdtype, device=self.device)
        grads = None
        if want_grads:
            f32 = dict(dtype=torch.float32, device=self.device)
            grads = dict(W_x=torch.empty(tuple(self.W_x.shape), **f32), b_x=torch.empty(tuple(self.b_x.shape), **f32),
                         W_h=torch.empty(tuple(self.W_h.shape), **f32), b_h=torch.empty(tuple(self.b_h.shape), **f32))
            if self.peep is not None:
                grads["peep"] = torch.empty(tuple(self.peep.shape), **f32)
        st = adjoint(self.prob, self.w, self.x, self.h0, h, g, self.ws, lam, dx, dh0, grads, check)
        return st, dict(lam=lam, dx=dx, dh0=dh0, **({} if grads is None else {"d" + k: v for k, v in grads.items()}))
