"""Thin Python binding of libfalcon (ctypes).

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI declared in ``include/falcon.h``.  Tensors must be
contiguous device tensors; outputs are allocated with torch when not given.
There is no CPU fallback: without the built library, or without a GPU,
these functions raise.
"""

from __future__ import annotations

import ctypes
import os
from typing import NamedTuple, Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfalcon.so")

VARIANTS = {"falcon1": 1, "falcon1a": 2, "falcon2": 3, "falcon2a": 4}
DTYPES = {torch.float32: 0, torch.bfloat16: 1}

FALCON_OK = 0


class FalconProblem(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("H", ctypes.c_int32), ("T", ctypes.c_int32),
                ("dk", ctypes.c_int32), ("dv", ctypes.c_int32), ("variant", ctypes.c_int32),
                ("io_dtype", ctypes.c_int32), ("eps", ctypes.c_float), ("eps_gamma", ctypes.c_float)]


class FalconConvProblem(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("C", ctypes.c_int32), ("W", ctypes.c_int32),
                ("io_dtype", ctypes.c_int32), ("activation", ctypes.c_int32), ("x_row", ctypes.c_int64)]


class FalconNormProblem(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("G", ctypes.c_int32), ("d", ctypes.c_int32),
                ("io_dtype", ctypes.c_int32), ("activation", ctypes.c_int32), ("center", ctypes.c_int32),
                ("x_heads", ctypes.c_int32), ("y_heads", ctypes.c_int32), ("eps", ctypes.c_float),
                ("scale", ctypes.c_float), ("x_row", ctypes.c_int64)]


class FalconScanProblem(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("D", ctypes.c_int32), ("N", ctypes.c_int32),
                ("G", ctypes.c_int32), ("io_dtype", ctypes.c_int32), ("softplus", ctypes.c_int32),
                ("x_row", ctypes.c_int64), ("dt_row", ctypes.c_int64), ("z_row", ctypes.c_int64),
                ("b_row", ctypes.c_int64), ("c_row", ctypes.c_int64)]


class FalconLinearProblem(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("H", ctypes.c_int32), ("T", ctypes.c_int32), ("dk", ctypes.c_int32),
                ("dv", ctypes.c_int32), ("io_dtype", ctypes.c_int32), ("qk_heads", ctypes.c_int32),
                ("v_heads", ctypes.c_int32), ("o_heads", ctypes.c_int32), ("scale", ctypes.c_float),
                ("q_row", ctypes.c_int64), ("k_row", ctypes.c_int64), ("v_row", ctypes.c_int64),
                ("zero_behind", ctypes.c_int32)]


class FalconResidualProblem(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("G", ctypes.c_int32), ("d", ctypes.c_int32),
                ("io_dtype", ctypes.c_int32), ("stream_dtype", ctypes.c_int32), ("activation", ctypes.c_int32),
                ("post_norm", ctypes.c_int32), ("pre_norm", ctypes.c_int32), ("eps", ctypes.c_float),
                ("y_row", ctypes.c_int64), ("gate_row", ctypes.c_int64), ("zero_behind", ctypes.c_int32)]


class FalconSavedPointers(ctypes.Structure):
    _fields_ = [("y_codes", ctypes.c_void_p), ("y_steps", ctypes.c_void_p), ("gate_codes", ctypes.c_void_p),
                ("gate_steps", ctypes.c_void_p)]


_P = ctypes.c_void_p
_SIGNATURES = {
    "falcon_abi_version": (ctypes.c_int32, []),
    "falcon_set_wait_limit": (ctypes.c_int32, [ctypes.c_int32]),
    "falcon_set_f1_launch_form": (ctypes.c_int32, [ctypes.c_int32]),
    "falcon_status_string": (ctypes.c_char_p, [ctypes.c_int32]),
    "falcon_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(FalconProblem), ctypes.c_int32]),
    "falcon_fwd_recurrent": (ctypes.c_int32, [ctypes.POINTER(FalconProblem), _P, _P, _P, _P, _P,
                                              _P, _P, _P, _P, _P]),
    "falcon_fwd_chunked": (ctypes.c_int32, [ctypes.POINTER(FalconProblem), _P, _P, _P, _P, _P, _P,
                                            _P, _P, _P, ctypes.c_int32, _P, ctypes.c_size_t, _P]),
    "falcon_fwd_chunked_noalloc": (ctypes.c_int32, [ctypes.POINTER(FalconProblem), _P, _P, _P, _P, _P,
                                                    _P, _P, _P, _P, ctypes.c_int32, _P]),
    "falcon_decode_step": (ctypes.c_int32, [ctypes.POINTER(FalconProblem), _P, _P, _P, _P, _P,
                                            _P, _P, _P, _P]),
    "falcon_bwd_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(FalconProblem)]),
    "falcon_bwd_chunked": (ctypes.c_int32, [ctypes.POINTER(FalconProblem)] + [_P] * 17
                           + [ctypes.c_size_t, _P]),
    "falcon_conv_fwd": (ctypes.c_int32, [ctypes.POINTER(FalconConvProblem)] + [_P] * 8),
    "falcon_conv_step": (ctypes.c_int32, [ctypes.POINTER(FalconConvProblem)] + [_P] * 7),
    "falcon_conv_bwd_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(FalconConvProblem)]),
    "falcon_conv_bwd": (ctypes.c_int32, [ctypes.POINTER(FalconConvProblem)] + [_P] * 6 + [ctypes.c_int32]
                        + [_P] * 6 + [ctypes.c_size_t, _P]),
    "falcon_norm_fwd": (ctypes.c_int32, [ctypes.POINTER(FalconNormProblem)] + [_P] * 5),
    "falcon_norm_bwd_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(FalconNormProblem)]),
    "falcon_norm_bwd": (ctypes.c_int32, [ctypes.POINTER(FalconNormProblem)] + [_P] * 4 + [ctypes.c_int32]
                        + [_P] * 4 + [ctypes.c_size_t, _P]),
    "falcon_scan_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(FalconScanProblem)]),
    "falcon_scan_fwd": (ctypes.c_int32, [ctypes.POINTER(FalconScanProblem)] + [_P] * 13 + [ctypes.c_size_t, _P]),
    "falcon_scan_step": (ctypes.c_int32, [ctypes.POINTER(FalconScanProblem)] + [_P] * 12),
    "falcon_scan_bwd_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(FalconScanProblem)]),
    "falcon_scan_bwd": (ctypes.c_int32, [ctypes.POINTER(FalconScanProblem)] + [_P] * 11 + [ctypes.c_int32]
                        + [_P] * 11 + [ctypes.c_size_t, _P]),
    "falcon_linear_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(FalconLinearProblem)]),
    "falcon_linear_fwd": (ctypes.c_int32, [ctypes.POINTER(FalconLinearProblem)] + [_P] * 9 + [ctypes.c_size_t, _P]),
    "falcon_linear_step": (ctypes.c_int32, [ctypes.POINTER(FalconLinearProblem)] + [_P] * 8),
    "falcon_linear_bwd_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(FalconLinearProblem)]),
    "falcon_linear_bwd": (ctypes.c_int32, [ctypes.POINTER(FalconLinearProblem)] + [_P] * 14 + [ctypes.c_size_t, _P]),
    "falcon_residual_fwd": (ctypes.c_int32, [ctypes.POINTER(FalconResidualProblem)] + [_P] * 9
                            + [ctypes.POINTER(FalconSavedPointers), _P]),
    "falcon_residual_bwd_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(FalconResidualProblem)]),
    "falcon_residual_bwd": (ctypes.c_int32, [ctypes.POINTER(FalconResidualProblem)] + [_P] * 2
                            + [ctypes.POINTER(FalconSavedPointers)] + [_P] * 6 + [ctypes.c_int32, _P, ctypes.c_int32]
                            + [_P] * 7 + [ctypes.c_size_t, _P]),
}

_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libfalcon.so (built by ``delta_rule_recurrence_amd.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m delta_rule_recurrence_amd.build`")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


class FalconError(RuntimeError):
    def __init__(self, status: int):
        self.status = status
        super().__init__(falcon_status_string(status))


def falcon_status_string(status: int) -> str:
    return load_library().falcon_status_string(int(status)).decode()


def falcon_abi_version() -> int:
    return int(load_library().falcon_abi_version())


def falcon_set_wait_limit(polls: int) -> int:
    """Polls a bounded wait between waves makes before giving up; returns the
    previous limit (see ``falcon_set_wait_limit`` in falcon.h)."""
    prev = int(load_library().falcon_set_wait_limit(int(polls)))
    if prev < 0:
        raise ValueError("the wait limit must be >= 0")
    return prev


F1_ONE_LAUNCH = 0
F1_TWO_LAUNCH = 1


def falcon_set_f1_launch_form(form: int) -> int:
    """How the Falcon-1 bf16 chunked fast path runs: F1_ONE_LAUNCH (default)
    or F1_TWO_LAUNCH; returns the previous form (see
    ``falcon_set_f1_launch_form`` in falcon.h)."""
    prev = int(load_library().falcon_set_f1_launch_form(int(form)))
    if prev < 0:
        raise ValueError("form must be F1_ONE_LAUNCH or F1_TWO_LAUNCH")
    return prev


def make_problem(B, H, T, dk, dv, *, variant="falcon1", io_dtype=torch.bfloat16, eps=1e-6,
                 eps_gamma=1e-6) -> FalconProblem:
    return FalconProblem(B, H, T, dk, dv, VARIANTS[variant], DTYPES[io_dtype], eps, eps_gamma)


def falcon_workspace_bytes(problem: FalconProblem, C: int) -> int:
    return int(load_library().falcon_workspace_bytes(ctypes.byref(problem), int(C)))


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a device tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return ctypes.c_void_p(t.data_ptr())


def _io_dtype(t: torch.Tensor, name: str) -> torch.dtype:
    if t.dtype not in DTYPES:
        raise ValueError(f"{name}: io dtype must be float32 or bfloat16, got {t.dtype}")
    return t.dtype


def _expect(t, name, shape, dtypes, device, *, optional=False):
    """Shape, dtype, device and layout check of one argument, done before any
    pointer crosses the C ABI (which cannot see shapes)."""
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype not in dtypes:
        names = " or ".join(str(d) for d in dtypes)
        raise ValueError(f"{name}: expected dtype {names}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")


def _expect_bytes(t, name, need, device):
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    have = t.numel() * t.element_size()
    if have < need:
        raise ValueError(f"{name}: {have} bytes, at least {need} needed")


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(status: int):
    if status != FALCON_OK:
        raise FalconError(status)


def _forward_setup(phi_k, phi_q, v, beta, lam, variant, S0, k_prev, o, S_T, return_state):
    """Checks every forward argument against the problem that phi_k and v
    define, and allocates the outputs that were not given."""
    if variant not in VARIANTS:
        raise ValueError(f"unknown variant {variant!r}")
    if not isinstance(phi_k, torch.Tensor) or phi_k.dim() != 4:
        raise ValueError("phi_k: expected a [B, H, T, dk] tensor")
    if not isinstance(v, torch.Tensor) or v.dim() != 4:
        raise ValueError("v: expected a [B, H, T, dv] tensor")
    B, H, T, dk = phi_k.shape
    dv = v.shape[-1]
    io = _io_dtype(v, "v")
    dev = v.device
    f32 = (torch.float32,)
    per_col = variant in ("falcon2", "falcon2a")
    _expect(phi_k, "phi_k", (B, H, T, dk), (io,), dev)
    _expect(phi_q, "phi_q", (B, H, T, dk), (io,), dev)
    _expect(v, "v", (B, H, T, dv), (io,), dev)
    _expect(beta, "beta", (B, H, T, dv) if per_col else (B, H, T), f32, dev)
    _expect(lam, "lam", (B, H, T), f32, dev)
    _expect(S0, "S0", (B, H, dk, dv), f32, dev, optional=True)
    _expect(k_prev, "k_prev", (B, H, dk), (io,), dev, optional=True)
    _expect(o, "o", (B, H, T, dv), (io,), dev, optional=True)
    _expect(S_T, "S_T", (B, H, dk, dv), f32, dev, optional=True)
    if o is None:
        o = torch.empty((B, H, T, dv), dtype=io, device=dev)
    if S_T is None and return_state:
        S_T = torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev)
    return B, H, T, dk, dv, o, S_T


def falcon_fwd_recurrent(phi_k, phi_q, v, beta, lam, *, variant="falcon1", S0=None, k_prev=None,
                         eps=1e-6, eps_gamma=1e-6, o=None, S_T=None, return_state=True,
                         stream=None):
    """Recurrent form; returns ``(o, S_T)``."""
    B, H, T, dk, dv, o, S_T = _forward_setup(phi_k, phi_q, v, beta, lam, variant, S0, k_prev, o,
                                             S_T, return_state)
    p = make_problem(B, H, T, dk, dv, variant=variant, io_dtype=v.dtype, eps=eps, eps_gamma=eps_gamma)
    _check(load_library().falcon_fwd_recurrent(
        ctypes.byref(p), _ptr(phi_k), _ptr(phi_q), _ptr(v), _ptr(beta), _ptr(lam), _ptr(S0),
        _ptr(k_prev), _ptr(o), _ptr(S_T), _stream(stream)))
    return o, S_T


def falcon_fwd_chunked(phi_k, phi_q, v, beta, lam, *, variant="falcon1", C=64, S0=None,
                       k_prev=None, eps=1e-6, eps_gamma=1e-6, o=None, S_T=None, workspace=None,
                       return_state=True, stream=None):
    """Chunk-parallel form; returns ``(o, S_T)``."""
    B, H, T, dk, dv, o, S_T = _forward_setup(phi_k, phi_q, v, beta, lam, variant, S0, k_prev, o,
                                             S_T, return_state)
    p = make_problem(B, H, T, dk, dv, variant=variant, io_dtype=v.dtype, eps=eps, eps_gamma=eps_gamma)
    need = falcon_workspace_bytes(p, C)
    if need == ctypes.c_size_t(-1).value:
        raise FalconError(-2 if C in (16, 32, 64) else -4)
    _expect_bytes(workspace, "workspace", need, v.device)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=v.device)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load_library().falcon_fwd_chunked(
        ctypes.byref(p), _ptr(phi_k), _ptr(phi_q), _ptr(v), _ptr(beta), _ptr(lam), _ptr(S0),
        _ptr(k_prev), _ptr(o), _ptr(S_T), int(C), _ptr(workspace), wbytes, _stream(stream)))
    return o, S_T


def falcon_fwd_chunked_noalloc(phi_k, phi_q, v, beta, lam, o, *, variant="falcon1", C=64, S0=None,
                               k_prev=None, eps=1e-6, eps_gamma=1e-6, S_T=None, stream=None):
    """Chunk-parallel form without any allocation: the caller passes ``o``
    (and ``S_T``, or None to skip the final state); scratch comes from the
    library's static device buffer.  Returns ``(o, S_T)``."""
    if o is None:
        raise ValueError("o is required: this entry point allocates nothing")
    B, H, T, dk, dv, o, S_T = _forward_setup(phi_k, phi_q, v, beta, lam, variant, S0, k_prev, o,
                                             S_T, False)
    p = make_problem(B, H, T, dk, dv, variant=variant, io_dtype=v.dtype, eps=eps, eps_gamma=eps_gamma)
    _check(load_library().falcon_fwd_chunked_noalloc(
        ctypes.byref(p), _ptr(phi_k), _ptr(phi_q), _ptr(v), _ptr(beta), _ptr(lam), _ptr(S0),
        _ptr(k_prev), _ptr(o), _ptr(S_T), int(C), _stream(stream)))
    return o, S_T


def falcon_decode_step(phi_k_prev, phi_q, v, beta, lam, S, *, variant="falcon1", is_first=None,
                       eps=1e-6, eps_gamma=1e-6, o=None, stream=None):
    """One decode token; updates ``S`` in place and returns ``o``."""
    if variant not in VARIANTS:
        raise ValueError(f"unknown variant {variant!r}")
    if not isinstance(phi_k_prev, torch.Tensor) or phi_k_prev.dim() != 3:
        raise ValueError("phi_k_prev: expected a [B, H, dk] tensor")
    if not isinstance(v, torch.Tensor) or v.dim() != 3:
        raise ValueError("v: expected a [B, H, dv] tensor")
    B, H, dk = phi_k_prev.shape
    dv = v.shape[-1]
    io = _io_dtype(v, "v")
    dev = v.device
    f32 = (torch.float32,)
    per_col = variant in ("falcon2", "falcon2a")
    _expect(phi_k_prev, "phi_k_prev", (B, H, dk), (io,), dev)
    _expect(phi_q, "phi_q", (B, H, dk), (io,), dev)
    _expect(v, "v", (B, H, dv), (io,), dev)
    _expect(beta, "beta", (B, H, dv) if per_col else (B, H), f32, dev)
    _expect(lam, "lam", (B, H), f32, dev)
    _expect(S, "S", (B, H, dk, dv), f32, dev)
    _expect(is_first, "is_first", (B,), (torch.uint8, torch.bool), dev, optional=True)
    _expect(o, "o", (B, H, dv), (io,), dev, optional=True)
    if o is None:
        o = torch.empty((B, H, dv), dtype=v.dtype, device=v.device)
    p = make_problem(B, H, 1, dk, dv, variant=variant, io_dtype=v.dtype, eps=eps, eps_gamma=eps_gamma)
    _check(load_library().falcon_decode_step(
        ctypes.byref(p), _ptr(phi_k_prev), _ptr(phi_q), _ptr(v), _ptr(beta), _ptr(lam), _ptr(S),
        _ptr(is_first), _ptr(o), _stream(stream)))
    return o


def falcon_bwd_workspace_bytes(problem: FalconProblem) -> int:
    return int(load_library().falcon_bwd_workspace_bytes(ctypes.byref(problem)))


def falcon_bwd_chunked(phi_k, phi_q, v, beta, lam, dO, *, S0=None, k_prev=None, dS_T=None,
                       eps=1e-6, eps_gamma=1e-6, grads=None, workspace=None, stream=None):
    """Gradients of ``<dO, o> + <dS_T, S_T>`` for the Falcon-1 forward.

    Returns a dict with float32 tensors dphi_k, dphi_q, dv, dbeta, dlam, dS0
    and dk_prev (None when ``k_prev`` is None).  ``grads`` may hold
    preallocated outputs under the same names.
    """
    B, H, T, dk, dv_, _, _ = _forward_setup(phi_k, phi_q, v, beta, lam, "falcon1", S0, k_prev,
                                            None, None, False)
    dev = v.device
    f32 = torch.float32
    _expect(dO, "dO", (B, H, T, dv_), (v.dtype,), dev)
    _expect(dS_T, "dS_T", (B, H, dk, dv_), (f32,), dev, optional=True)
    shapes = {"dphi_k": (B, H, T, dk), "dphi_q": (B, H, T, dk), "dv": (B, H, T, dv_),
              "dbeta": (B, H, T), "dlam": (B, H, T), "dS0": (B, H, dk, dv_), "dk_prev": (B, H, dk)}
    g = dict(grads or {})
    unknown = set(g) - set(shapes)
    if unknown:
        raise ValueError(f"grads: unknown names {sorted(unknown)}")
    for name, shape in shapes.items():
        _expect(g.get(name), f"grads[{name!r}]", shape, (f32,), dev, optional=True)
        if g.get(name) is None and (name != "dk_prev" or k_prev is not None):
            g[name] = torch.empty(shape, dtype=f32, device=dev)
    if k_prev is None:
        g["dk_prev"] = None
    p = make_problem(B, H, T, dk, dv_, variant="falcon1", io_dtype=v.dtype, eps=eps,
                     eps_gamma=eps_gamma)
    need = falcon_bwd_workspace_bytes(p)
    if need == ctypes.c_size_t(-1).value:
        raise FalconError(-2)
    _expect_bytes(workspace, "workspace", need, dev)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load_library().falcon_bwd_chunked(
        ctypes.byref(p), _ptr(phi_k), _ptr(phi_q), _ptr(v), _ptr(beta), _ptr(lam), _ptr(S0),
        _ptr(k_prev), _ptr(dO), _ptr(dS_T), _ptr(g["dphi_k"]), _ptr(g["dphi_q"]), _ptr(g["dv"]),
        _ptr(g["dbeta"]), _ptr(g["dlam"]), _ptr(g["dS0"]), _ptr(g["dk_prev"]), _ptr(workspace),
        wbytes, _stream(stream)))
    return g


# ---- around the recurrence: short convolution, group norm, selective scan,
#      linear attention, residual update --------------------------------------------
#
# Channels-last "rows" inputs ([B, T, width], or [B, width] for single tokens)
# may be some of the columns of a wider contiguous projection; everything else
# is contiguous.  The calls run on ``stream`` (default: the current stream of
# the inputs' device); what they allocate belongs to that stream.

ACTIVATIONS = {"none": 0, "silu": 1, "elu1": 2}
GATES = {"none": 0, "silu": 1, "sigmoid": 3}
_LAYOUTS = ("rows", "heads")
_F32 = (torch.float32,)


def _is(t, shape, dtype, device):
    """Whether t is a contiguous tensor of this shape, type and device."""
    return (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype == dtype and t.device == device
            and t.is_contiguous())


def _need(t, name, shape, dtype, device, *, optional=False):
    """``_expect`` for one type, quick where all is well."""
    if not (_is(t, shape, dtype, device) or (optional and t is None)):
        _expect(t, name, shape, (dtype,), device, optional=optional)


def _row_step(t, name, shape, dtype, device, tail=1):
    """Checks a rows tensor ([..., width], the last ``tail`` axes dense) and
    returns the elements from one row to the next."""
    if _is(t, shape, dtype, device):
        return shape[-1] if tail == 1 else shape[-1] * shape[-2]
    if isinstance(t, torch.Tensor) and t.shape == shape and t.dtype == dtype and t.device == device:
        # columns of a contiguous projection, the usual case
        stride, width = t.stride(), shape[-1]
        if stride[-1] == 1 and (tail == 1 or (stride[-2] == width and shape[-1] > 1)):
            width = width if tail == 1 else width * shape[-2]
            row = stride[-tail - 1]
            if row >= width and min(shape) > 1 and (len(shape) == tail + 1 or stride[0] == row * shape[1]):
                return row
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: expected dtype {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    width = _count(shape[-tail:])
    stride = t.stride()
    lead = len(shape) - tail
    dense = 1
    for axis in range(len(shape) - 1, lead - 1, -1):
        if shape[axis] != 1 and stride[axis] != dense:
            raise ValueError(f"{name}: the last {tail} axes must be dense")
        dense *= shape[axis]
    # rows one step apart: every leading axis continues the one below it
    row = next((stride[axis] // _count(shape[axis + 1:lead]) for axis in range(lead) if shape[axis] != 1), width)
    for axis in range(lead):
        if shape[axis] != 1 and stride[axis] != row * _count(shape[axis + 1:lead]):
            raise ValueError(f"{name}: rows must be evenly spaced (columns of one contiguous projection)")
    if row < width:
        raise ValueError(f"{name}: rows overlap")
    return row


def _count(sizes):
    n = 1
    for size in sizes:
        n *= size
    return n


def _activation(name, allowed):
    if name not in allowed:
        raise ValueError(f"unknown activation {name!r}: expected one of {sorted(allowed)}")
    return ACTIVATIONS[name]


# The current stream's handle without the Stream object around it (2.7 us of a
# small call's 12), where torch has the call.
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda index: torch.cuda.current_stream(index).cuda_stream)


class _On:
    """Makes a device and, if given, a stream current for one call."""

    def __init__(self, device, stream):
        self._within = [torch.cuda.device(device)] + ([torch.cuda.stream(stream)] if stream is not None else [])
        self._of = device

    def __enter__(self):
        for w in self._within:
            w.__enter__()
        return torch.cuda.current_stream(self._of).cuda_stream

    def __exit__(self, *exc):
        for w in reversed(self._within):
            w.__exit__(*exc)
        return False


class _Here:
    """The stream that is current already."""

    def __init__(self, stream):
        self._stream = stream

    def __enter__(self):
        return self._stream

    def __exit__(self, *exc):
        return False


def _on_stream(device, stream):
    """The device and stream of one call: allocations and the launch use them."""
    if device.type != "cuda":
        raise ValueError("expected a device tensor")
    if stream is None and device.index == torch.cuda.current_device():
        return _Here(_current_stream(device.index))
    if stream is not None and stream.device != device:
        raise ValueError(f"stream: on {stream.device}, the inputs are on {device}")
    return _On(device, stream)


def _ref(t):
    """Address of a checked tensor, or NULL."""
    return None if t is None else t.data_ptr()


def _workspace(given, need, device):
    """The given workspace or a new one, and its size."""
    if need == ctypes.c_size_t(-1).value:
        raise FalconError(-2)
    _expect_bytes(given, "workspace", need, device)
    if given is None and need > 0:
        given = torch.empty(need, dtype=torch.uint8, device=device)
    return given, (0 if given is None else given.numel() * given.element_size())


def _new(shape, dtype, device, lengths=None):
    """An output; zeros behind the sequences' ends, which calls leave alone."""
    return (torch.empty if lengths is None else torch.zeros)(shape, dtype=dtype, device=device)


def _grads(given, shapes, device):
    """Checked gradients by name; those not given are allocated by the caller."""
    g = dict(given or {})
    unknown = set(g) - set(shapes)
    if unknown:
        raise ValueError(f"grads: unknown names {sorted(unknown)}")
    for name, t in g.items():
        _expect(t, f"grads[{name!r}]", shapes[name], _F32, device, optional=True)
    return g


def _allocate(g, shapes, wanted, device):
    """The gradients that are wanted and not given; None for the others.  (A second
    tensor of a shape costs 1.2 us, a first one 1.8 of a small call's 20.)"""
    made = {}
    for name, shape in shapes.items():
        if g.get(name) is None:
            if not wanted[name]:
                g[name] = None
            elif shape in made:
                g[name] = torch.empty_like(made[shape])
            else:
                made[shape] = g[name] = torch.empty(shape, dtype=torch.float32, device=device)


def _dy_dtype(dy, shape, device):
    if not isinstance(dy, torch.Tensor):
        raise TypeError(f"dy: expected a torch.Tensor, got {type(dy).__name__}")
    _expect(dy, "dy", shape, tuple(DTYPES), device)
    return DTYPES[dy.dtype]


def _conv_setup(x, weight, bias, activation, dims):
    act = _activation(activation, ("none", "silu"))
    if not isinstance(x, torch.Tensor) or x.dim() != dims:
        raise ValueError("x: expected a [B, T, C] tensor" if dims == 3 else "x: expected a [B, C] tensor")
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight: expected a [C, W] tensor")
    io, dev, C, W = _io_dtype(x, "x"), x.device, x.shape[-1], weight.shape[1]
    _need(weight, "weight", (C, W), torch.float32, dev)
    _need(bias, "bias", (C,), torch.float32, dev, optional=True)
    row = _row_step(x, "x", x.shape, io, dev)
    T = x.shape[1] if dims == 3 else 1
    return io, dev, W, FalconConvProblem(x.shape[0], T, C, W, DTYPES[io], act, row)


def falcon_conv_fwd(x, weight, bias=None, *, activation="silu", state=None, lengths=None, y=None,
                    state_out=None, return_state=False, stream=None):
    """Short causal convolution of ``x [B, T, C]`` with ``weight [C, W]``
    (W in 2, 3, 4) and an activation ("silu" or "none"); returns
    ``(y, state_out)``.

    ``state`` holds the W - 1 rows before the first token (``[B, W - 1, C]``,
    default zero); ``state_out`` (given, or allocated with ``return_state``)
    gets the last W - 1 up to each sequence's end.  ``lengths`` (``[B]`` int32)
    marks padded sequences: rows of ``y`` behind the end stay as they were, or
    zero when ``y`` is allocated here.
    """
    io, dev, W, p = _conv_setup(x, weight, bias, activation, 3)
    B, T, C = x.shape
    _need(state, "state", (B, W - 1, C), io, dev, optional=True)
    _need(lengths, "lengths", (B,), torch.int32, dev, optional=True)
    _need(y, "y", (B, T, C), io, dev, optional=True)
    _need(state_out, "state_out", (B, W - 1, C), io, dev, optional=True)
    with _on_stream(dev, stream) as st:
        if y is None:
            y = _new((B, T, C), io, dev, lengths)
        if state_out is None and return_state:
            state_out = torch.empty((B, W - 1, C), dtype=io, device=dev)
        _check(load_library().falcon_conv_fwd(ctypes.byref(p), _ref(x), _ref(weight), _ref(bias), _ref(state),
                                              _ref(lengths), _ref(y), _ref(state_out), st))
    return y, state_out


def falcon_conv_step(x, weight, state, bias=None, *, activation="silu", is_first=None, y=None, stream=None):
    """One token ``x [B, C]`` of every sequence; moves ``state [B, W - 1, C]``
    on in place and returns ``y [B, C]``.  ``is_first`` (``[B]`` bytes) marks
    sequences whose earlier rows count as zero."""
    io, dev, W, p = _conv_setup(x, weight, bias, activation, 2)
    B, C = x.shape
    _need(state, "state", (B, W - 1, C), io, dev)
    _expect(is_first, "is_first", (B,), (torch.uint8, torch.bool), dev, optional=True)
    _need(y, "y", (B, C), io, dev, optional=True)
    with _on_stream(dev, stream) as st:
        if y is None:
            y = torch.empty((B, C), dtype=io, device=dev)
        _check(load_library().falcon_conv_step(ctypes.byref(p), _ref(x), _ref(weight), _ref(bias), _ref(state),
                                               _ref(is_first), _ref(y), st))
    return y


def falcon_conv_bwd_workspace_bytes(problem: FalconConvProblem) -> int:
    return int(load_library().falcon_conv_bwd_workspace_bytes(ctypes.byref(problem)))


def falcon_conv_bwd(x, weight, dy, bias=None, *, activation="silu", state=None, lengths=None, dstate_out=None,
                    grads=None, workspace=None, stream=None):
    """Gradients of ``<dy, y> + <dstate_out, state_out>``: a dict of float32
    tensors dx (zero behind the sequences' ends), dweight, dbias (None without
    a bias) and dstate (None without a state, unless ``grads`` holds one)."""
    io, dev, W, p = _conv_setup(x, weight, bias, activation, 3)
    B, T, C = x.shape
    _need(state, "state", (B, W - 1, C), io, dev, optional=True)
    _need(lengths, "lengths", (B,), torch.int32, dev, optional=True)
    _need(dstate_out, "dstate_out", (B, W - 1, C), torch.float32, dev, optional=True)
    dy_dtype = _dy_dtype(dy, (B, T, C), dev)
    shapes = {"dx": (B, T, C), "dweight": (C, W), "dbias": (C,), "dstate": (B, W - 1, C)}
    g = _grads(grads, shapes, dev)
    need = falcon_conv_bwd_workspace_bytes(p)
    wanted = {"dx": True, "dweight": True, "dbias": bias is not None, "dstate": state is not None}
    _expect_bytes(workspace, "workspace", 0 if need == ctypes.c_size_t(-1).value else need, dev)
    with _on_stream(dev, stream) as st:
        for name, shape in shapes.items():
            if g.get(name) is None:
                g[name] = torch.empty(shape, dtype=torch.float32, device=dev) if wanted[name] else None
        workspace, have = _workspace(workspace, need, dev)
        _check(load_library().falcon_conv_bwd(
            ctypes.byref(p), _ref(x), _ref(weight), _ref(bias), _ref(state), _ref(lengths), _ref(dy), dy_dtype,
            _ref(dstate_out), _ref(g["dx"]), _ref(g["dweight"]), _ref(g["dbias"]), _ref(g["dstate"]),
            _ref(workspace), have, st))
    return g


def _norm_setup(x, groups, weight, bias, center, activation, eps, scale, x_layout, y_layout):
    act = _activation(activation, tuple(ACTIVATIONS))
    for name, layout in (("x_layout", x_layout), ("y_layout", y_layout)):
        if layout not in _LAYOUTS:
            raise ValueError(f"{name}: expected \"rows\" or \"heads\", got {layout!r}")
    heads = x_layout == "heads"
    if not isinstance(x, torch.Tensor) or x.dim() != (4 if heads else 3):
        raise ValueError("x: expected a [B, G, T, d] tensor" if heads else "x: expected a [B, T, C] tensor")
    G = int(groups)
    if G < 1 or (x.shape[1] != G if heads else x.shape[2] % G != 0):
        raise ValueError(f"groups: {groups} does not divide x of shape {tuple(x.shape)}")
    io, dev = _io_dtype(x, "x"), x.device
    B, T = x.shape[0], x.shape[2] if heads else x.shape[1]
    d = x.shape[3] if heads else x.shape[2] // G
    if heads:
        _need(x, "x", (B, G, T, d), io, dev)
    row = G * d if heads else _row_step(x, "x", x.shape, io, dev)
    _need(weight, "weight", (G * d,), torch.float32, dev, optional=True)
    _need(bias, "bias", (G * d,), torch.float32, dev, optional=True)
    rows, by_head = (B, T, G * d), (B, G, T, d)
    p = FalconNormProblem(B, T, G, d, DTYPES[io], act, int(bool(center)), int(heads), int(y_layout == "heads"),
                          eps, scale, row)
    return io, dev, p, (by_head if y_layout == "heads" else rows)


def falcon_norm_fwd(x, groups, weight=None, bias=None, *, center=False, activation="none", eps=1e-6, scale=1.0,
                    x_layout="rows", y_layout="rows", y=None, stream=None):
    """Group norm with an activation, a token's group (head) of d channels at a
    time: ``scale * f(weight * xhat + bias)``, with ``xhat`` the group over its
    root mean square (``center``: less its mean, over its deviation).

    ``x`` and ``y`` are ``[B, T, G d]`` ("rows") or ``[B, G, T, d]`` ("heads",
    the layout of the recurrences); ``activation`` is "none", "silu" or "elu1"
    (elu + 1, a positive feature map); ``weight`` and ``bias`` are ``[G d]``.
    """
    io, dev, p, y_shape = _norm_setup(x, groups, weight, bias, center, activation, eps, scale, x_layout, y_layout)
    _need(y, "y", y_shape, io, dev, optional=True)
    with _on_stream(dev, stream) as st:
        if y is None:
            y = torch.empty(y_shape, dtype=io, device=dev)
        _check(load_library().falcon_norm_fwd(ctypes.byref(p), _ref(x), _ref(weight), _ref(bias), _ref(y), st))
    return y


def falcon_norm_bwd_workspace_bytes(problem: FalconNormProblem) -> int:
    return int(load_library().falcon_norm_bwd_workspace_bytes(ctypes.byref(problem)))


def falcon_norm_bwd(x, groups, dy, weight=None, bias=None, *, center=False, activation="none", eps=1e-6, scale=1.0,
                    x_layout="rows", y_layout="rows", grads=None, workspace=None, stream=None):
    """Gradients of ``<dy, y>``: a dict of float32 tensors dx (x's layout),
    dweight and dbias (None where weight or bias is None, unless ``grads``
    holds them).  ``dy`` has y's layout."""
    io, dev, p, y_shape = _norm_setup(x, groups, weight, bias, center, activation, eps, scale, x_layout, y_layout)
    dy_dtype = _dy_dtype(dy, y_shape, dev)
    C = p.G * p.d
    shapes = {"dx": tuple(x.shape), "dweight": (C,), "dbias": (C,)}
    g = _grads(grads, shapes, dev)
    need = falcon_norm_bwd_workspace_bytes(p)
    wanted = {"dx": True, "dweight": weight is not None, "dbias": bias is not None}
    _expect_bytes(workspace, "workspace", 0 if need == ctypes.c_size_t(-1).value else need, dev)
    with _on_stream(dev, stream) as st:
        for name, shape in shapes.items():
            if g.get(name) is None:
                g[name] = torch.empty(shape, dtype=torch.float32, device=dev) if wanted[name] else None
        workspace, have = _workspace(workspace, need, dev)
        _check(load_library().falcon_norm_bwd(
            ctypes.byref(p), _ref(x), _ref(weight), _ref(bias), _ref(dy), dy_dtype, _ref(g["dx"]),
            _ref(g["dweight"]), _ref(g["dbias"]), _ref(workspace), have, st))
    return g


def _scan_setup(x, dt, A, B, C, D, dt_bias, softplus, z, dims):
    if not isinstance(x, torch.Tensor) or x.dim() != dims:
        raise ValueError("x: expected a [B, T, D] tensor" if dims == 3 else "x: expected a [B, D] tensor")
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise ValueError("A: expected a [D, N] tensor")
    if not isinstance(B, torch.Tensor) or B.dim() != dims + 1:
        raise ValueError("B: expected a [B, T, G, N] tensor" if dims == 3 else "B: expected a [B, G, N] tensor")
    io, dev, width, N, G = _io_dtype(x, "x"), x.device, x.shape[-1], A.shape[1], B.shape[-2]
    _need(A, "A", (width, N), torch.float32, dev)
    _need(D, "D", (width,), torch.float32, dev, optional=True)
    _need(dt_bias, "dt_bias", (width,), torch.float32, dev, optional=True)
    shared = tuple(x.shape[:-1]) + (G, N)
    rows = [_row_step(x, "x", x.shape, io, dev), _row_step(dt, "dt", x.shape, io, dev),
            _row_step(z, "z", x.shape, io, dev) if z is not None else width,
            _row_step(B, "B", shared, io, dev, 2), _row_step(C, "C", shared, io, dev, 2)]
    p = FalconScanProblem(x.shape[0], x.shape[1] if dims == 3 else 1, width, N, G, DTYPES[io], int(bool(softplus)), *rows)
    return io, dev, p


def falcon_scan_workspace_bytes(problem: FalconScanProblem) -> int:
    return int(load_library().falcon_scan_workspace_bytes(ctypes.byref(problem)))


def falcon_scan_fwd(x, dt, A, B, C, *, D=None, dt_bias=None, softplus=True, z=None, S0=None, lengths=None, y=None,
                    S_T=None, workspace=None, return_state=True, stream=None):
    """Selective state space scan of ``x, dt [B, T, D]`` with ``A [D, N]``
    (N in 8, 16, 32, 64) and ``B, C [B, T, G, N]``; returns ``(y, S_T)``.

    ``S_t = exp(delta_t A) S_(t-1) + delta_t x_t B_t`` and
    ``y_t = (<C_t, S_t> + D x_t) silu(z_t)``, with ``delta = softplus(dt +
    dt_bias)`` (or without the softplus) and the gate only where ``z`` is given.
    ``S0`` and ``S_T`` are ``[B, D, N]`` float32; ``lengths`` (``[B]`` int32)
    marks padded sequences: ``S_T`` is the state at the end, rows of ``y``
    behind it stay as they were, or zero when ``y`` is allocated here.
    """
    io, dev, p = _scan_setup(x, dt, A, B, C, D, dt_bias, softplus, z, 3)
    nb, T, width = x.shape
    state = (nb, width, p.N)
    _need(S0, "S0", state, torch.float32, dev, optional=True)
    _need(lengths, "lengths", (nb,), torch.int32, dev, optional=True)
    _need(y, "y", (nb, T, width), io, dev, optional=True)
    _need(S_T, "S_T", state, torch.float32, dev, optional=True)
    need = falcon_scan_workspace_bytes(p)
    _expect_bytes(workspace, "workspace", 0 if need == ctypes.c_size_t(-1).value else need, dev)
    with _on_stream(dev, stream) as st:
        if y is None:
            y = _new((nb, T, width), io, dev, lengths)
        if S_T is None and return_state:
            S_T = torch.empty(state, dtype=torch.float32, device=dev)
        workspace, have = _workspace(workspace, need, dev)
        _check(load_library().falcon_scan_fwd(
            ctypes.byref(p), _ref(x), _ref(dt), _ref(A), _ref(B), _ref(C), _ref(D), _ref(dt_bias), _ref(z), _ref(S0),
            _ref(lengths), _ref(y), _ref(S_T), _ref(workspace), have, st))
    return y, S_T


def falcon_scan_step(x, dt, A, B, C, S, *, D=None, dt_bias=None, softplus=True, z=None, is_first=None, y=None,
                     stream=None):
    """One token of every sequence (``x, dt, z [B, D]``, ``B, C [B, G, N]``);
    moves ``S [B, D, N]`` on in place and returns ``y [B, D]``.  ``is_first``
    (``[B]`` bytes) marks sequences whose state so far counts as zero."""
    io, dev, p = _scan_setup(x, dt, A, B, C, D, dt_bias, softplus, z, 2)
    nb, width = x.shape
    _need(S, "S", (nb, width, p.N), torch.float32, dev)
    _expect(is_first, "is_first", (nb,), (torch.uint8, torch.bool), dev, optional=True)
    _need(y, "y", (nb, width), io, dev, optional=True)
    with _on_stream(dev, stream) as st:
        if y is None:
            y = torch.empty((nb, width), dtype=io, device=dev)
        _check(load_library().falcon_scan_step(
            ctypes.byref(p), _ref(x), _ref(dt), _ref(A), _ref(B), _ref(C), _ref(D), _ref(dt_bias), _ref(z), _ref(S),
            _ref(is_first), _ref(y), st))
    return y


def falcon_scan_bwd_workspace_bytes(problem: FalconScanProblem) -> int:
    return int(load_library().falcon_scan_bwd_workspace_bytes(ctypes.byref(problem)))


def falcon_scan_bwd(x, dt, A, B, C, dy, *, D=None, dt_bias=None, softplus=True, z=None, S0=None, lengths=None,
                    dS_T=None, grads=None, workspace=None, stream=None):
    """Gradients of ``<dy, y> + <dS_T, S_T>``: a dict of float32 tensors dx,
    ddt, dA, dB, dC, dD, ddt_bias, dz and dS0; dD, ddt_bias, dz and dS0 are
    None where D, dt_bias, z or S0 is None (all but dz may still be asked for
    through ``grads``).  Rows behind the sequences' ends get zero."""
    io, dev, p = _scan_setup(x, dt, A, B, C, D, dt_bias, softplus, z, 3)
    nb, T, width = x.shape
    state, shared = (nb, width, p.N), (nb, T, p.G, p.N)
    _need(S0, "S0", state, torch.float32, dev, optional=True)
    _need(lengths, "lengths", (nb,), torch.int32, dev, optional=True)
    _need(dS_T, "dS_T", state, torch.float32, dev, optional=True)
    dy_dtype = _dy_dtype(dy, (nb, T, width), dev)
    shapes = {"dx": (nb, T, width), "ddt": (nb, T, width), "dz": (nb, T, width), "dA": (width, p.N), "dB": shared,
              "dC": shared, "dD": (width,), "ddt_bias": (width,), "dS0": state}
    g = _grads(grads, shapes, dev)
    if z is None and g.get("dz") is not None:
        raise ValueError("grads['dz']: there is no z")
    missing = {"dz": z is None, "dD": D is None, "ddt_bias": dt_bias is None, "dS0": S0 is None}
    need = falcon_scan_bwd_workspace_bytes(p)
    _expect_bytes(workspace, "workspace", 0 if need == ctypes.c_size_t(-1).value else need, dev)
    with _on_stream(dev, stream) as st:
        for name, shape in shapes.items():
            if g.get(name) is None:
                g[name] = None if missing.get(name) else torch.empty(shape, dtype=torch.float32, device=dev)
        workspace, have = _workspace(workspace, need, dev)
        _check(load_library().falcon_scan_bwd(
            ctypes.byref(p), _ref(x), _ref(dt), _ref(A), _ref(B), _ref(C), _ref(D), _ref(dt_bias), _ref(z), _ref(S0),
            _ref(lengths), _ref(dy), dy_dtype, _ref(dS_T), _ref(g["dx"]), _ref(g["ddt"]), _ref(g["dz"]), _ref(g["dA"]),
            _ref(g["dB"]), _ref(g["dC"]), _ref(g["dD"]), _ref(g["ddt_bias"]), _ref(g["dS0"]), _ref(workspace), have, st))
    return g


def _by_head(t, name, layout, shape, io, dev):
    """Checks a tensor of heads ([B, H, T, d], ``shape``) in either layout;
    elements from one row to the next."""
    B, H, T, d = shape
    if layout == "heads":
        _need(t, name, shape, io, dev)
        return H * d
    return _row_step(t, name, (B, T, H * d), io, dev)


def _laid(layout, B, H, T, d):
    return (B, H, T, d) if layout == "heads" else (B, T, H * d)


def _linear_setup(q, k, v, log_decay, scale, qk_layout, v_layout, o_layout):
    for name, layout in (("qk_layout", qk_layout), ("v_layout", v_layout), ("o_layout", o_layout)):
        if layout not in _LAYOUTS:
            raise ValueError(f"{name}: expected \"rows\" or \"heads\", got {layout!r}")
    if not isinstance(log_decay, torch.Tensor) or log_decay.dim() != 1 or log_decay.shape[0] < 1:
        raise ValueError("log_decay: expected an [H] tensor")
    H = log_decay.shape[0]
    sizes = []
    for name, t, layout in (("q", q, qk_layout), ("v", v, v_layout)):
        heads = layout == "heads"
        if not isinstance(t, torch.Tensor) or t.dim() != (4 if heads else 3):
            raise ValueError(f"{name}: expected a [B, H, T, d] tensor" if heads else f"{name}: expected a [B, T, H d] tensor")
        if t.shape[1] != H if heads else t.shape[2] % H != 0:
            raise ValueError(f"{name}: {H} heads do not fit its shape {tuple(t.shape)}")
        sizes.append((t.shape[0], H, *t.shape[2:]) if heads else (t.shape[0], H, t.shape[1], t.shape[2] // H))
    B, H, T, dk = sizes[0]
    dv = sizes[1][3]
    io, dev = _io_dtype(q, "q"), q.device
    _need(log_decay, "log_decay", (H,), torch.float32, dev)
    rows = [_by_head(q, "q", qk_layout, (B, H, T, dk), io, dev), _by_head(k, "k", qk_layout, (B, H, T, dk), io, dev),
            _by_head(v, "v", v_layout, (B, H, T, dv), io, dev)]
    return io, dev, FalconLinearProblem(B, H, T, dk, dv, DTYPES[io], int(qk_layout == "heads"), int(v_layout == "heads"),
                                        int(o_layout == "heads"), scale, *rows)


def falcon_linear_workspace_bytes(problem: FalconLinearProblem) -> int:
    return int(load_library().falcon_linear_workspace_bytes(ctypes.byref(problem)))


def falcon_linear_fwd(q, k, v, log_decay, *, scale=1.0, S0=None, lengths=None, qk_layout="heads", v_layout="heads",
                      o_layout="heads", o=None, S_T=None, workspace=None, return_state=True, stream=None):
    """Linear attention with a decay for each head (``log_decay [H]``, at most
    zero); returns ``(o, S_T)``.

    ``S_t = exp(log_decay) S_(t-1) + k_t v_t'`` and ``o_t = scale S_t' q_t``.
    ``q`` and ``k``, ``v`` and ``o`` are each ``[B, H, T, d]`` ("heads") or
    ``[B, T, H d]`` ("rows"), with d in 16, 32, 64, 128.  ``S0`` and ``S_T`` are
    ``[B, H, dk, dv]`` float32; ``lengths`` (``[B]`` int32) marks padded
    sequences: ``S_T`` is the state at the end, rows of ``o`` behind it stay as
    they were, or zero when ``o`` is allocated here.
    """
    io, dev, p = _linear_setup(q, k, v, log_decay, scale, qk_layout, v_layout, o_layout)
    state, out = (p.B, p.H, p.dk, p.dv), _laid(o_layout, p.B, p.H, p.T, p.dv)
    _need(S0, "S0", state, torch.float32, dev, optional=True)
    _need(lengths, "lengths", (p.B,), torch.int32, dev, optional=True)
    _need(o, "o", out, io, dev, optional=True)
    _need(S_T, "S_T", state, torch.float32, dev, optional=True)
    need = falcon_linear_workspace_bytes(p)
    _expect_bytes(workspace, "workspace", 0 if need == ctypes.c_size_t(-1).value else need, dev)
    with _on_stream(dev, stream) as st:
        if o is None:
            o = torch.empty(out, dtype=io, device=dev)
            p.zero_behind = 1
        if S_T is None and return_state:
            S_T = torch.empty(state, dtype=torch.float32, device=dev)
        workspace, have = _workspace(workspace, need, dev)
        _check(load_library().falcon_linear_fwd(
            ctypes.byref(p), _ref(q), _ref(k), _ref(v), _ref(log_decay), _ref(S0), _ref(lengths), _ref(o), _ref(S_T),
            _ref(workspace), have, st))
    return o, S_T


def falcon_linear_step(q, k, v, log_decay, S, *, scale=1.0, is_first=None, o=None, stream=None):
    """One token of every sequence (``q, k [B, H, dk]``, ``v [B, H, dv]``); moves
    ``S [B, H, dk, dv]`` on in place and returns ``o [B, H, dv]``.  ``is_first``
    (``[B]`` bytes) marks sequences whose state so far counts as zero."""
    for name, t in (("q", q), ("v", v)):
        if not isinstance(t, torch.Tensor) or t.dim() != 3:
            raise ValueError(f"{name}: expected a [B, H, d] tensor")
    B, H, dk = q.shape
    dv = v.shape[2]
    io, dev = _io_dtype(q, "q"), q.device
    rows = [_row_step(t, name, (B, H, d), io, dev, 2) for t, name, d in ((q, "q", dk), (k, "k", dk), (v, "v", dv))]
    _need(log_decay, "log_decay", (H,), torch.float32, dev)
    _need(S, "S", (B, H, dk, dv), torch.float32, dev)
    _expect(is_first, "is_first", (B,), (torch.uint8, torch.bool), dev, optional=True)
    _need(o, "o", (B, H, dv), io, dev, optional=True)
    p = FalconLinearProblem(B, H, 1, dk, dv, DTYPES[io], 0, 0, 0, scale, *rows)
    with _on_stream(dev, stream) as st:
        if o is None:
            o = torch.empty((B, H, dv), dtype=io, device=dev)
        _check(load_library().falcon_linear_step(ctypes.byref(p), _ref(q), _ref(k), _ref(v), _ref(log_decay), _ref(S),
                                                 _ref(is_first), _ref(o), st))
    return o


def falcon_linear_bwd_workspace_bytes(problem: FalconLinearProblem) -> int:
    return int(load_library().falcon_linear_bwd_workspace_bytes(ctypes.byref(problem)))


def falcon_linear_bwd(q, k, v, log_decay, dO, *, scale=1.0, S0=None, lengths=None, dS_T=None, learned_decay=False,
                      qk_layout="heads", v_layout="heads", o_layout="heads", grads=None, workspace=None, stream=None):
    """Gradients of ``<dO, o> + <dS_T, S_T>``: a dict of float32 tensors dq, dk
    and dv (in the layouts of q, k and v; zero behind the sequences' ends), dS0
    (None without an S0) and dlog_decay (None unless ``learned_decay``); either
    of the last two may still be asked for through ``grads``.  ``dO`` has o's
    layout and type."""
    io, dev, p = _linear_setup(q, k, v, log_decay, scale, qk_layout, v_layout, o_layout)
    state = (p.B, p.H, p.dk, p.dv)
    _need(S0, "S0", state, torch.float32, dev, optional=True)
    _need(lengths, "lengths", (p.B,), torch.int32, dev, optional=True)
    _need(dO, "dO", _laid(o_layout, p.B, p.H, p.T, p.dv), io, dev)
    _need(dS_T, "dS_T", state, torch.float32, dev, optional=True)
    by_qk, by_v = _laid(qk_layout, p.B, p.H, p.T, p.dk), _laid(v_layout, p.B, p.H, p.T, p.dv)
    shapes = {"dq": by_qk, "dk": by_qk, "dv": by_v, "dlog_decay": (p.H,), "dS0": state}
    g = _grads(grads, shapes, dev)
    wanted = {"dq": True, "dk": True, "dv": True, "dlog_decay": learned_decay, "dS0": S0 is not None}
    need = falcon_linear_bwd_workspace_bytes(p)
    _expect_bytes(workspace, "workspace", 0 if need == ctypes.c_size_t(-1).value else need, dev)
    with _on_stream(dev, stream) as st:
        _allocate(g, shapes, wanted, dev)
        workspace, have = _workspace(workspace, need, dev)
        _check(load_library().falcon_linear_bwd(
            ctypes.byref(p), _ref(q), _ref(k), _ref(v), _ref(log_decay), _ref(S0), _ref(lengths), _ref(dO), _ref(dS_T),
            _ref(g["dq"]), _ref(g["dk"]), _ref(g["dv"]), _ref(g["dlog_decay"]), _ref(g["dS0"]), _ref(workspace), have, st))
    return g


class FalconSaved(NamedTuple):
    """A block's output and gate in 8 bits: codes ``[B, T, C]`` int8 and, for every
    32 channels, the exponent of their step, ``[B, T, ceil(C / 32)]`` uint8."""

    y_codes: torch.Tensor
    y_steps: torch.Tensor
    gate_codes: Optional[torch.Tensor] = None
    gate_steps: Optional[torch.Tensor] = None


def _saved(saved, rows, gated, dev):
    """Checks the tensors in 8 bits of [B, T, C] ``rows`` and returns their pointers."""
    if not isinstance(saved, tuple) or len(saved) != 4:
        raise TypeError(f"saved: expected a FalconSaved, got {type(saved).__name__}")
    steps = rows[:2] + ((rows[2] + 31) // 32,)
    for name, t, shape, dtype in zip(FalconSaved._fields, saved, (rows, steps) * 2, (torch.int8, torch.uint8) * 2):
        if gated or not name.startswith("gate"):
            _need(t, name, shape, dtype, dev)
    return FalconSavedPointers(*(_ref(t) if gated or i < 2 else None for i, t in enumerate(saved)))


def _incoming(t, name, rows, dev):
    """``_expect`` for a gradient of either type, quick where all is well."""
    if not (isinstance(t, torch.Tensor) and t.dtype in DTYPES and _is(t, rows, t.dtype, dev)):
        _expect(t, name, rows, tuple(DTYPES), dev)


def _residual_weights(C, dev, **weights):
    for name, t in weights.items():
        if t is not None:
            _need(t, name, (C,), torch.float32, dev)


def _groups(groups, C):
    G = int(groups)
    if G < 1 or C % G != 0:
        raise ValueError(f"groups: {groups} does not divide {C} channels")
    return G


def _gate_activation(activation):
    if activation not in GATES:
        raise ValueError(f"unknown activation {activation!r}: expected one of {sorted(GATES)}")
    return GATES[activation]


def falcon_residual_fwd(y, h=None, *, gate=None, activation="silu", groups=1, post_norm=True, post_weight=None,
                        alpha=None, pre_norm=True, pre_weight=None, eps=1e-6, lengths=None, h_out=None, n=None,
                        save=False, saved=None, stream=None):
    """From a block's output ``y [B, T, C]`` to the next block's input; returns
    ``(h_out, n, saved)``.

    ``h_out = h + alpha f(gate) z`` with ``z`` the groups of ``y`` over their root
    mean squares, times ``post_weight`` (``post_norm`` false: ``y`` itself), and ``n``
    the rows of ``h_out`` over theirs, times ``pre_weight`` (``pre_norm`` false:
    None).  ``activation`` is "silu", "sigmoid" or "none"; weights and ``alpha`` are
    ``[C]`` float32; ``h`` and ``h_out``, the stream, may be of another type than
    ``y``, and ``h_out`` may be ``h``.  ``save`` (or a FalconSaved to fill) keeps
    ``y`` and ``gate`` in 8 bits for the backward pass.  ``lengths`` (``[B]`` int32)
    marks padded sequences: rows behind the end stay as they were, or zero where they
    are allocated here.
    """
    act = _gate_activation(activation)
    if not isinstance(y, torch.Tensor) or y.dim() != 3:
        raise ValueError("y: expected a [B, T, C] tensor")
    io, dev, rows = _io_dtype(y, "y"), y.device, tuple(y.shape)
    B, T, C = rows
    G = _groups(groups, C)
    y_row = _row_step(y, "y", y.shape, io, dev)
    gate_row = _row_step(gate, "gate", y.shape, io, dev) if gate is not None else C
    kind = h if h is not None else h_out
    stream_type = _io_dtype(kind, "h") if isinstance(kind, torch.Tensor) else io
    _need(h, "h", rows, stream_type, dev, optional=True)
    _need(h_out, "h_out", rows, stream_type, dev, optional=True)
    _need(n, "n", rows, io, dev, optional=True)
    if n is not None and not pre_norm:
        raise ValueError("n: there is no pre_norm")
    _residual_weights(C, dev, post_weight=post_weight, alpha=alpha, pre_weight=pre_weight)
    _need(lengths, "lengths", (B,), torch.int32, dev, optional=True)
    p = FalconResidualProblem(B, T, G, C // G, DTYPES[io], DTYPES[stream_type], act, int(bool(post_norm)),
                              int(bool(pre_norm)), eps, y_row, gate_row)
    with _on_stream(dev, stream) as st:
        # rows behind the ends: cleared by the call, but where some outputs are given and others not
        p.zero_behind = h_out is None and n is None and saved is None
        fill = None if p.zero_behind else lengths
        if h_out is None:
            h_out = _new(rows, stream_type, dev, fill) if fill is not None or h is None else torch.empty_like(h)
        if n is None and pre_norm:
            n = _new(rows, io, dev, fill) if fill is not None or stream_type != io else torch.empty_like(h_out)
        at = None
        if saved is not None:
            at = ctypes.byref(_saved(saved, rows, gate is not None, dev))
        elif save:
            pair = [_new(rows, torch.int8, dev, fill), _new((B, T, (C + 31) // 32), torch.uint8, dev, fill)]
            if gate is not None:
                pair += [torch.empty_like(t) if fill is None else torch.zeros_like(t) for t in pair]
            saved = FalconSaved(*pair)
            at = ctypes.byref(FalconSavedPointers(*map(_ref, saved)))
        _check(load_library().falcon_residual_fwd(
            ctypes.byref(p), _ref(y), _ref(gate), _ref(h), _ref(post_weight), _ref(alpha), _ref(pre_weight),
            _ref(lengths), _ref(h_out), _ref(n), at, st))
    return h_out, n, saved


def falcon_residual_bwd_workspace_bytes(problem: FalconResidualProblem) -> int:
    return int(load_library().falcon_residual_bwd_workspace_bytes(ctypes.byref(problem)))


def falcon_residual_bwd(y, h_out, dh_out, dn=None, *, gate=None, saved=None, activation="silu", groups=1,
                        post_norm=True, post_weight=None, alpha=None, pre_norm=True, pre_weight=None, eps=1e-6,
                        lengths=None, added=True, grads=None, workspace=None, stream=None):
    """Gradients of ``<dh_out, h_out> + <dn, n>``: a dict of float32 tensors dy, dgate
    (None without a gate), dh (None unless ``added``: there was an ``h``), dalpha,
    dpost_weight and dpre_weight (None where alpha or the weight is None); all but the
    first two may still be asked for through ``grads``, the weights' where there is the
    norm.  ``saved`` holds ``y`` and ``gate`` in 8 bits; both are None then.  ``h_out`` and ``dn`` belong to
    ``pre_norm``; ``dh_out`` may be None (zero).  Rows behind the sequences' ends get
    zero."""
    act = _gate_activation(activation)
    if saved is not None:
        if y is not None or gate is not None:
            raise ValueError("saved: y and gate are in it")
        lead = saved[0] if isinstance(saved, tuple) and len(saved) == 4 else None
    else:
        lead = y
    if not isinstance(lead, torch.Tensor) or lead.dim() != 3:
        raise ValueError("saved: expected a FalconSaved of [B, T, C] codes" if saved is not None else "y: expected a [B, T, C] tensor")
    dev, rows = lead.device, tuple(lead.shape)
    B, T, C = rows
    G = _groups(groups, C)
    y_row = gate_row = C
    io, at = torch.float32, None
    if saved is not None:
        gated = saved[2] is not None
        at = _saved(saved, rows, gated, dev)
    else:
        io, gated = _io_dtype(y, "y"), gate is not None
        y_row = _row_step(y, "y", y.shape, io, dev)
        gate_row = _row_step(gate, "gate", y.shape, io, dev) if gated else C
    stream_type = torch.float32
    if pre_norm:
        stream_type = _io_dtype(h_out, "h_out") if isinstance(h_out, torch.Tensor) else None
        _need(h_out, "h_out", rows, stream_type, dev)
        _incoming(dn, "dn", rows, dev)
    elif h_out is not None or dn is not None:
        raise ValueError("h_out, dn: there is no pre_norm")
    if dh_out is not None:
        _incoming(dh_out, "dh_out", rows, dev)
    _residual_weights(C, dev, post_weight=post_weight, alpha=alpha, pre_weight=pre_weight)
    _need(lengths, "lengths", (B,), torch.int32, dev, optional=True)
    shapes = {"dy": rows, "dgate": rows, "dh": rows, "dalpha": (C,), "dpost_weight": (C,), "dpre_weight": (C,)}
    g = _grads(grads, shapes, dev)
    for name, there in (("dgate", gated), ("dpost_weight", post_norm), ("dpre_weight", pre_norm)):
        if g.get(name) is not None and not there:
            raise ValueError(f"grads[{name!r}]: there is no {'gate' if name == 'dgate' else name[1:-7] + '_norm'}")
    wanted = {"dy": True, "dgate": gated, "dh": added, "dalpha": alpha is not None,
              "dpost_weight": post_norm and post_weight is not None, "dpre_weight": pre_norm and pre_weight is not None}
    p = FalconResidualProblem(B, T, G, C // G, DTYPES[io], DTYPES[stream_type], act, int(bool(post_norm)),
                              int(bool(pre_norm)), eps, y_row, gate_row)
    need = falcon_residual_bwd_workspace_bytes(p)
    _expect_bytes(workspace, "workspace", 0 if need == ctypes.c_size_t(-1).value else need, dev)
    types = [DTYPES[t.dtype] if t is not None else 0 for t in (dh_out, dn)]
    with _on_stream(dev, stream) as st:
        _allocate(g, shapes, wanted, dev)
        workspace, have = _workspace(workspace, need, dev)
        _check(load_library().falcon_residual_bwd(
            ctypes.byref(p), _ref(y), _ref(gate), None if at is None else ctypes.byref(at), _ref(h_out),
            _ref(post_weight), _ref(alpha), _ref(pre_weight), _ref(lengths), _ref(dh_out), types[0], _ref(dn), types[1],
            _ref(g["dy"]), _ref(g["dgate"]), _ref(g["dh"]), _ref(g["dalpha"]), _ref(g["dpost_weight"]),
            _ref(g["dpre_weight"]), _ref(workspace), have, st))
    return g
