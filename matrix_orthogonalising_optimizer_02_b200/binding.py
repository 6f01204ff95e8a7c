"""Thin Python binding of ``include/muon_b200.h`` (ctypes).

Argument marshalling only: every step of the path runs in ``libmuon_b200.so``.
Tensors are passed by ``data_ptr()``; the stream defaults to torch's current
CUDA stream.  There is no fallback: if the library is not built, or a call
fails, a ``MuonError`` is raised.
"""
from __future__ import annotations

import array
import ctypes
import itertools
import os
from ctypes import POINTER, c_double, c_float, c_int, c_longlong, c_size_t, c_void_p
from dataclasses import dataclass
from typing import Optional, Sequence

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmuon_b200.so")

# enums of muon_b200.h
MUON_OK, MUON_ERR_INVALID_ARG, MUON_ERR_UNSUPPORTED_SHAPE, MUON_ERR_ALIGNMENT = 0, 1, 2, 3
MUON_ERR_WORKSPACE_TOO_SMALL, MUON_ERR_CUDA, MUON_ERR_NONFINITE, MUON_ERR_DEVICE_TIMEOUT = 4, 5, 6, 7
MUON_ERR_DEVICE_UNDRAINED = 8
MUON_BF16, MUON_F32, MUON_F16 = 0, 1, 2
SCALE_MODES = {"moonlight": 0, "kellerjordan": 1, "mup": 2, "naive": 3}
MUON_MAX_NS_ITERS = 32
KERNEL_KINDS = {"momentum": 0, "scale": 1, "ns_gemm": 2, "update": 3, "simt_gemm": 4, "lu": 5, "misc": 6,
                "tc_f32": 7, "simt_gemm_f64": 8, "grad_norm": 9, "adamw": 10}

#: Exported entry points, as declared in include/muon_b200.h.
EXPORTED = (
    "muon_step_workspace_size", "muon_step_workspace_min", "muon_step_batched",
    "ns_workspace_size", "ns_orthogonalize", "stiefel_workspace_size", "stiefel_cayley_step",
    "muon_workspace_device_status", "muon_timing_enable", "muon_timing_reset", "muon_timing_read",
    "muon_status_string", "muon_build_info", "muon_frobenius_prescale_static",
    "muon_cayley_workspace_size", "muon_cayley_step", "muon_step_host_grad_workspace_size",
    "muon_step_batched_host_grad", "muon_last_error", "muon_selftest_wait_timeout",
    "ns_stacks_workspace_size", "ns_stacks_saved_size", "ns_orthogonalize_stacks",
    "ns_stacks_backward_workspace_size", "ns_orthogonalize_stacks_backward",
    "muon_stacks_workspace_size", "muon_step_stacks",
    "grad_norm_workspace_size", "grad_norm_batched", "adamw_step_batched",
)


class MuonError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib().muon_status_string(status).decode() if _LIB is not None else str(status)
        if status == MUON_ERR_CUDA and _LIB is not None:
            detail = _LIB.muon_last_error()
            if detail:
                msg += f": {detail.decode()}"
        super().__init__(f"{where}: {msg} (status {status})")


class NsSchedule(ctypes.Structure):
    _fields_ = [("n_iters", c_int), ("coeffs", POINTER(c_float)), ("n_split_iters", c_int),
                ("fp32_mode", c_int), ("eps", c_float)]


class MatrixDesc(ctypes.Structure):
    _fields_ = [("W", c_void_p), ("G", c_void_p), ("M", c_void_p), ("O_out", c_void_p),
                ("rows", c_int), ("cols", c_int), ("w_dtype", c_int), ("g_dtype", c_int)]


class Hyper(ctypes.Structure):
    _fields_ = [("lr", c_float), ("beta", c_float), ("weight_decay", c_float), ("nesterov", c_int),
                ("scale_mode", c_int), ("ns", NsSchedule)]


class NsStackDesc(ctypes.Structure):
    _fields_ = [("X", c_void_p), ("Y", c_void_p), ("x_stride", c_longlong), ("y_stride", c_longlong),
                ("x_ld", c_int), ("y_ld", c_int), ("count", c_int), ("rows", c_int), ("cols", c_int),
                ("x_dtype", c_int), ("y_dtype", c_int)]


class MuonStackDesc(ctypes.Structure):
    _fields_ = [("W", c_void_p), ("G", c_void_p), ("M", c_void_p),
                ("w_stride", c_longlong), ("g_stride", c_longlong), ("m_stride", c_longlong),
                ("w_ld", c_int), ("g_ld", c_int), ("m_ld", c_int), ("count", c_int), ("rows", c_int), ("cols", c_int),
                ("w_dtype", c_int), ("g_dtype", c_int)]


class AdamWTensorDesc(ctypes.Structure):
    _fields_ = [("W", c_void_p), ("G", c_void_p), ("m", c_void_p), ("v", c_void_p), ("n", c_longlong),
                ("w_dtype", c_int), ("g_dtype", c_int)]


class AdamWHyper(ctypes.Structure):
    _fields_ = [("lr", c_double), ("beta1", c_double), ("beta2", c_double), ("eps", c_double),
                ("weight_decay", c_double), ("step", c_longlong), ("step_dev", c_void_p)]


_LIB = None


def _lib():
    global _LIB
    if _LIB is not None:
        return _LIB
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run `python -m matrix_orthogonalising_optimizer_02_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    sig = {
        "muon_step_workspace_size": (c_size_t, [POINTER(MatrixDesc), c_int, POINTER(Hyper)]),
        "muon_step_workspace_min": (c_size_t, [POINTER(MatrixDesc), c_int, POINTER(Hyper)]),
        "muon_step_batched": (c_int, [POINTER(MatrixDesc), c_int, POINTER(Hyper), c_void_p, c_size_t, c_void_p]),
        "muon_step_host_grad_workspace_size": (c_size_t, [POINTER(MatrixDesc), c_int, POINTER(Hyper)]),
        "muon_step_batched_host_grad": (c_int, [POINTER(MatrixDesc), c_int, POINTER(Hyper), c_void_p, c_size_t,
                                                c_void_p]),
        "ns_workspace_size": (c_size_t, [c_int, c_int, c_int, POINTER(NsSchedule)]),
        "ns_orthogonalize": (c_int, [c_void_p, c_int, c_void_p, c_int, c_int, c_int, c_int, POINTER(NsSchedule),
                                     c_void_p, c_size_t, c_void_p]),
        "stiefel_workspace_size": (c_size_t, [c_int, c_int, c_int]),
        "stiefel_cayley_step": (c_int, [c_void_p, c_void_p, c_int, c_int, c_int, c_float, c_void_p, c_size_t,
                                        c_void_p]),
        "muon_workspace_device_status": (c_int, [c_void_p, c_size_t, POINTER(c_int), c_void_p]),
        "muon_timing_enable": (c_int, [c_int]),
        "muon_timing_reset": (c_int, []),
        "muon_timing_read": (c_int, [c_int, POINTER(c_double), POINTER(c_longlong), POINTER(c_double)]),
        "muon_status_string": (ctypes.c_char_p, [c_int]),
        "muon_last_error": (ctypes.c_char_p, []),
        "muon_selftest_wait_timeout": (c_int, [c_void_p, c_size_t, c_void_p]),
        "muon_build_info": (ctypes.c_char_p, []),
        "muon_cayley_workspace_size": (c_size_t, [c_int, c_int, c_int]),
        "muon_cayley_step": (c_int, [c_void_p, c_void_p, c_void_p, c_int, c_int, c_int, c_float, c_float, c_int,
                                     c_void_p, c_size_t, c_void_p]),
        "muon_frobenius_prescale_static": (c_int, [c_void_p, c_int, c_void_p, c_int, c_int, c_int, c_int, c_int,
                                                   c_float, c_void_p, c_void_p]),
        "ns_stacks_workspace_size": (c_size_t, [POINTER(NsStackDesc), c_int, POINTER(NsSchedule), c_int]),
        "ns_stacks_saved_size": (c_size_t, [POINTER(NsStackDesc), c_int, POINTER(NsSchedule)]),
        "ns_orthogonalize_stacks": (c_int, [POINTER(NsStackDesc), c_int, POINTER(NsSchedule), c_void_p, c_size_t,
                                            c_void_p, c_size_t, c_void_p]),
        "ns_stacks_backward_workspace_size": (c_size_t, [POINTER(NsStackDesc), c_int, POINTER(NsSchedule)]),
        "ns_orthogonalize_stacks_backward": (c_int, [POINTER(NsStackDesc), c_int, POINTER(NsSchedule), c_void_p,
                                                     c_size_t, c_void_p, c_size_t, c_void_p]),
        "muon_stacks_workspace_size": (c_size_t, [POINTER(MuonStackDesc), c_int, POINTER(Hyper)]),
        "muon_step_stacks": (c_int, [POINTER(MuonStackDesc), c_int, POINTER(Hyper), c_void_p, c_void_p, c_size_t,
                                     c_void_p]),
        "grad_norm_workspace_size": (c_size_t, [POINTER(AdamWTensorDesc), c_int]),
        "grad_norm_batched": (c_int, [POINTER(AdamWTensorDesc), c_int, c_float, c_void_p, c_void_p, c_size_t,
                                      c_void_p]),
        "adamw_step_batched": (c_int, [POINTER(AdamWTensorDesc), c_int, POINTER(AdamWHyper), c_void_p, c_void_p]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name, None)
        if fn is None:       # reported by the export test; calling it raises AttributeError
            continue
        fn.restype = res
        fn.argtypes = args
    _LIB = lib
    return lib


def load():
    """Loads the shared library (raises if it is missing) and returns the ctypes handle."""
    return _lib()


def _check(status: int, where: str):
    if status != MUON_OK:
        raise MuonError(status, where)


def _stream(stream) -> int:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return MUON_BF16
    if t.dtype == torch.float32:
        return MUON_F32
    raise TypeError(f"unsupported dtype {t.dtype}: bf16 or fp32 expected")


class Schedule:
    """Newton-Schulz schedule: per-iteration (a, b, c), split-bf16 prefix, fp32 mode, eps."""

    def __init__(self, coeffs: Sequence[Sequence[float]], n_split_iters: int = 0, fp32_mode: bool = False,
                 eps: float = 1e-7):
        flat = [float(x) for abc in coeffs for x in abc]
        self._arr = (c_float * max(1, len(flat)))(*flat)
        self.c = NsSchedule(len(coeffs), ctypes.cast(self._arr, POINTER(c_float)), int(n_split_iters),
                            int(bool(fp32_mode)), float(eps))
        self.coeffs = [tuple(abc) for abc in coeffs]

    @classmethod
    def fixed(cls, steps: int = 5, coeffs=(3.4445, -4.7750, 2.0315), **kw):
        return cls([coeffs] * steps, **kw)

    @classmethod
    def hybrid(cls, n_fast: int = 8, n_stable: int = 2, fast=(3.4445, -4.7750, 2.0315),
               stable=(1.875, -1.25, 0.375), **kw):
        return cls([fast] * n_fast + [stable] * n_stable, **kw)


@dataclass
class Matrix:
    """One Muon matrix: W (bf16/fp32, updated in place), G (bf16/fp32), M (fp32, updated in
    place), optional O_out receiving the Newton-Schulz output."""
    W: object
    G: object
    M: object
    O_out: Optional[object] = None


def _need(t, name: str, cuda: bool = True, device=None):
    """Checks a tensor handed to the library by its data pointer: dense (a strided view's
    pointer would be read as another matrix) and on the expected device."""
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (the library reads it as a dense row-major array)")
    if cuda and not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if cuda and device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _descs(mats: Sequence[Matrix], g_on_host: bool = False):
    import torch
    arr = (MatrixDesc * len(mats))()
    for i, m in enumerate(mats):
        if m.W.dim() != 2:
            raise ValueError("W must be a 2-D matrix")
        rows, cols = m.W.shape
        if tuple(m.G.shape) != (rows, cols) or tuple(m.M.shape) != (rows, cols):
            raise ValueError("W, G and M must have the same 2-D shape")
        if m.M.dtype != torch.float32:
            raise TypeError("the momentum buffer M must be fp32")
        _need(m.W, "W")
        _need(m.M, "M", device=m.W.device)
        _need(m.G, "G", cuda=not g_on_host, device=m.W.device)
        if m.O_out is not None:
            if tuple(m.O_out.shape) != (rows, cols):
                raise ValueError("O_out must have W's shape")
            _need(m.O_out, "O_out", device=m.W.device)
        arr[i] = MatrixDesc(m.W.data_ptr(), m.G.data_ptr(), m.M.data_ptr(),
                            m.O_out.data_ptr() if m.O_out is not None else None,
                            rows, cols, _dtype_code(m.W), _dtype_code(m.G))
    return arr


def hyper(lr: float, beta: float = 0.95, weight_decay: float = 0.0, nesterov: bool = False,
          scale_mode: str = "moonlight", schedule: Optional[Schedule] = None) -> tuple:
    sch = schedule if schedule is not None else Schedule.fixed(5)
    h = Hyper(float(lr), float(beta), float(weight_decay), int(bool(nesterov)), SCALE_MODES[scale_mode], sch.c)
    return (h, sch)   # keep the schedule (and its coefficient array) alive with the struct


def muon_step_workspace_size(mats: Sequence[Matrix], hp) -> int:
    return int(_lib().muon_step_workspace_size(_descs(mats), len(mats), ctypes.byref(hp[0])))


def muon_step_workspace_min(mats: Sequence[Matrix], hp) -> int:
    return int(_lib().muon_step_workspace_min(_descs(mats), len(mats), ctypes.byref(hp[0])))


def muon_step_batched(mats: Sequence[Matrix], hp, workspace, stream=None):
    st = _lib().muon_step_batched(_descs(mats), len(mats), ctypes.byref(hp[0]), workspace.data_ptr(),
                                  workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "muon_step_batched")


def muon_step_host_grad_workspace_size(mats: Sequence[Matrix], hp) -> int:
    return int(_lib().muon_step_host_grad_workspace_size(_descs(mats, g_on_host=True), len(mats),
                                                         ctypes.byref(hp[0])))


def muon_step_batched_host_grad(mats: Sequence[Matrix], hp, workspace, stream=None):
    """muon_step_batched with every G a pinned CPU tensor: the library streams the gradients
    in chunk by chunk, overlapping the copies with the step of earlier chunks."""
    for m in mats:
        if m.G.is_cuda or not m.G.is_pinned():
            raise ValueError("G must be a pinned CPU tensor (tensor.pin_memory())")
    st = _lib().muon_step_batched_host_grad(_descs(mats, g_on_host=True), len(mats), ctypes.byref(hp[0]),
                                            workspace.data_ptr(),
                                            workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "muon_step_batched_host_grad")


def ns_workspace_size(batch: int, rows: int, cols: int, schedule: Schedule) -> int:
    return int(_lib().ns_workspace_size(batch, rows, cols, ctypes.byref(schedule.c)))


def ns_orthogonalize(X_in, X_out, schedule: Schedule, workspace, stream=None):
    _need(X_in, "X_in")
    _need(X_out, "X_out", device=X_in.device)
    if X_in.dim() == 2:
        batch, (rows, cols) = 1, X_in.shape
    else:
        batch, rows, cols = X_in.shape
    if tuple(X_out.shape) != tuple(X_in.shape):
        raise ValueError("X_out must have X_in's shape")
    if not (X_in.is_contiguous() and X_out.is_contiguous()):
        raise ValueError("X_in and X_out must be contiguous")
    st = _lib().ns_orthogonalize(X_in.data_ptr(), _dtype_code(X_in), X_out.data_ptr(), _dtype_code(X_out),
                                 batch, rows, cols, ctypes.byref(schedule.c), workspace.data_ptr(),
                                 workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "ns_orthogonalize")


def stiefel_workspace_size(batch: int, n: int, k: int) -> int:
    return int(_lib().stiefel_workspace_size(batch, n, k))


def stiefel_cayley_step(W, G, lr: float, workspace, stream=None):
    _need(W, "W")
    _need(G, "G", device=W.device)
    if W.dim() == 2:
        batch, (n, k) = 1, W.shape
    else:
        batch, n, k = W.shape
    if tuple(G.shape) != tuple(W.shape):
        raise ValueError("G must have W's shape")
    st = _lib().stiefel_cayley_step(W.data_ptr(), G.data_ptr(), batch, n, k, float(lr), workspace.data_ptr(),
                                    workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "stiefel_cayley_step")


def frobenius_prescale_static(X_in, X_out, fp32_mode: bool = False, eps: float = 1e-7, scale_out=None,
                              stream=None):
    """X_out = X0 / (||X0||_F + eps) per matrix without a workspace: the library's fixed
    internal scratch is used instead (see muon_frobenius_prescale_static in the header)."""
    _need(X_in, "X_in")
    _need(X_out, "X_out", device=X_in.device)
    if X_in.dim() == 2:
        batch, (rows, cols) = 1, X_in.shape
    else:
        batch, rows, cols = X_in.shape
    if tuple(X_out.shape) != tuple(X_in.shape):
        raise ValueError("X_out must have X_in's shape")
    st = _lib().muon_frobenius_prescale_static(X_in.data_ptr(), _dtype_code(X_in), X_out.data_ptr(),
                                               _dtype_code(X_out), batch, rows, cols, int(bool(fp32_mode)),
                                               float(eps), scale_out.data_ptr() if scale_out is not None else None,
                                               _stream(stream))
    _check(st, "muon_frobenius_prescale_static")


def muon_cayley_workspace_size(batch: int, n: int, k: int) -> int:
    return int(_lib().muon_cayley_workspace_size(batch, n, k))


def muon_cayley_step(W, G, M, lr: float, beta: float, workspace, center: bool = True, stream=None):
    _need(W, "W")
    _need(G, "G", device=W.device)
    _need(M, "M", device=W.device)
    if W.dim() == 2:
        batch, (n, k) = 1, W.shape
    else:
        batch, n, k = W.shape
    if tuple(G.shape) != tuple(W.shape) or tuple(M.shape) != tuple(W.shape):
        raise ValueError("G and M must have W's shape")
    st = _lib().muon_cayley_step(W.data_ptr(), G.data_ptr(), M.data_ptr(), batch, n, k, float(lr), float(beta),
                                 int(bool(center)), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                 _stream(stream))
    _check(st, "muon_cayley_step")


def device_status(workspace, stream=None) -> int:
    out = c_int(-1)
    st = _lib().muon_workspace_device_status(workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                             ctypes.byref(out), _stream(stream))
    _check(st, "muon_workspace_device_status")
    return out.value


def timing_enable(on: bool = True):
    _check(_lib().muon_timing_enable(int(bool(on))), "muon_timing_enable")


def timing_reset():
    _check(_lib().muon_timing_reset(), "muon_timing_reset")


def timing_read(kind: str):
    ms, n, work = c_double(), c_longlong(), c_double()
    _check(_lib().muon_timing_read(KERNEL_KINDS[kind], ctypes.byref(ms), ctypes.byref(n), ctypes.byref(work)),
           "muon_timing_read")
    return ms.value, n.value, work.value


def workspace(nbytes: int, device=None):
    """A caller-owned workspace tensor of at least nbytes (allocated by torch)."""
    import torch
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device or "cuda")


# ---------------------------------------------------------------------------- stacks of blocks
@dataclass
class Stack:
    """Blocks to orthogonalise: X and Y are [count, rows, cols] (or one [rows, cols]) views with a unit
    stride in the last dimension, bf16, fp16 or fp32 each.  Y may be X.  For the gradient, X is the
    gradient of the output and Y receives that of the input."""
    X: object
    Y: object


@dataclass
class MuonStack:
    """Blocks of a Muon parameter: W (updated in place), G and M (fp32, updated in place), each a
    [count, rows, cols] (or one [rows, cols]) view with a unit stride in the last dimension."""
    W: object
    G: object
    M: object


@dataclass
class AdamWTensor:
    """A dense tensor of any shape: W (updated in place), G, and the fp32 moments m and v."""
    W: object
    G: object
    m: object
    v: object


_CODES: dict = {}


def _codes() -> dict:
    """muon_dtype by torch dtype (filled on first use: the module imports without torch)."""
    if not _CODES:
        import torch
        _CODES.update({torch.bfloat16: MUON_BF16, torch.float32: MUON_F32, torch.float16: MUON_F16})
    return _CODES


def _dtype16(t, name: str) -> int:
    code = _codes().get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}: bf16, fp16 or fp32 expected")
    return code


def _view3(t, name: str, device):
    """(shape, row pitch, block stride) of a [count, rows, cols] or [rows, cols] view."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dim() not in (2, 3):
        raise ValueError(f"{name} must be [count, rows, cols] or [rows, cols], got shape {tuple(t.shape)}")
    shape = tuple(t.shape) if t.dim() == 3 else (1,) + tuple(t.shape)
    if 0 in shape:
        raise ValueError(f"{name} has no elements")
    stride = t.stride() if t.dim() == 3 else (0,) + t.stride()
    if shape[2] > 1 and stride[2] != 1:
        raise ValueError(f"{name} must have a unit stride in its last dimension")
    ld = stride[1] if shape[1] > 1 else shape[2]
    if ld >= 1 << 31:
        raise ValueError(f"{name}: row pitch {ld} is too long")
    return shape, ld, stride[0] if shape[0] > 1 else shape[1] * shape[2]


def _stack_descs(stacks: Sequence[Stack]):
    if not stacks:
        raise ValueError("no stacks")
    arr = (NsStackDesc * len(stacks))()
    device = stacks[0].X.device
    for i, s in enumerate(stacks):
        shape, x_ld, x_stride = _view3(s.X, "X", device)
        yshape, y_ld, y_stride = _view3(s.Y, "Y", device)
        if yshape != shape:
            raise ValueError("X and Y must have the same shape")
        arr[i] = NsStackDesc(s.X.data_ptr(), s.Y.data_ptr(), x_stride, y_stride, x_ld, y_ld, *shape,
                             _dtype16(s.X, "X"), _dtype16(s.Y, "Y"))
    return arr, device


def _muon_stack_descs(stacks: Sequence[MuonStack]):
    import torch
    if not stacks:
        raise ValueError("no stacks")
    arr = (MuonStackDesc * len(stacks))()
    device = stacks[0].W.device
    for i, s in enumerate(stacks):
        shape, w_ld, w_stride = _view3(s.W, "W", device)
        gshape, g_ld, g_stride = _view3(s.G, "G", device)
        mshape, m_ld, m_stride = _view3(s.M, "M", device)
        if gshape != shape or mshape != shape:
            raise ValueError("W, G and M must have the same shape")
        if s.M.dtype != torch.float32:
            raise TypeError("the momentum buffer M must be fp32")
        arr[i] = MuonStackDesc(s.W.data_ptr(), s.G.data_ptr(), s.M.data_ptr(), w_stride, g_stride, m_stride,
                               w_ld, g_ld, m_ld, *shape, _dtype16(s.W, "W"), _dtype16(s.G, "G"))
    return arr, device


def _bytes(t, name: str, device):
    _need(t, name, device=device)
    return t.data_ptr(), t.numel() * t.element_size()


def _scalar(t, name: str, device, dtype):
    """Pointer of a one-element device tensor (None: a null pointer)."""
    if t is None:
        return None
    if t.dtype != dtype or t.numel() != 1:
        raise ValueError(f"{name} must be one {dtype} value on the device")
    _need(t, name, device=device)
    return t.data_ptr()


class _On:
    """Makes the tensors' device the current one for a call and gives the stream: the caller's, or
    torch's current stream of that device."""

    def __init__(self, device, stream):
        import torch
        self.guard = torch.cuda.device(device) if device.index != torch.cuda.current_device() else None
        self.device, self.stream = device, stream

    def __enter__(self):
        import torch
        if self.guard is not None:
            self.guard.__enter__()
        return _stream(self.stream if self.stream is not None else torch.cuda.current_stream(self.device))

    def __exit__(self, *exc):
        return self.guard.__exit__(*exc) if self.guard is not None else None


def ns_stacks_workspace_size(stacks: Sequence[Stack], schedule: Schedule, with_saved: bool = False) -> int:
    return int(_lib().ns_stacks_workspace_size(_stack_descs(stacks)[0], len(stacks), ctypes.byref(schedule.c),
                                               int(bool(with_saved))))


def ns_stacks_saved_size(stacks: Sequence[Stack], schedule: Schedule) -> int:
    return int(_lib().ns_stacks_saved_size(_stack_descs(stacks)[0], len(stacks), ctypes.byref(schedule.c)))


def ns_orthogonalize_stacks(stacks: Sequence[Stack], schedule: Schedule, workspace, saved=None, stream=None):
    """Newton-Schulz orthogonalisation of every block; `saved` keeps what the gradient needs."""
    arr, device = _stack_descs(stacks)
    ws, ws_bytes = _bytes(workspace, "workspace", device)
    sv, sv_bytes = _bytes(saved, "saved", device) if saved is not None else (None, 0)
    with _On(device, stream) as st:
        _check(_lib().ns_orthogonalize_stacks(arr, len(stacks), ctypes.byref(schedule.c), sv, sv_bytes, ws, ws_bytes,
                                              st), "ns_orthogonalize_stacks")


def ns_stacks_backward_workspace_size(grads: Sequence[Stack], schedule: Schedule) -> int:
    return int(_lib().ns_stacks_backward_workspace_size(_stack_descs(grads)[0], len(grads), ctypes.byref(schedule.c)))


def ns_orthogonalize_stacks_backward(grads: Sequence[Stack], schedule: Schedule, saved, workspace, stream=None):
    """The gradient of ns_orthogonalize_stacks: X of each stack is the gradient of its output, Y
    receives that of its input; `saved` is the buffer the forward call filled."""
    arr, device = _stack_descs(grads)
    ws, ws_bytes = _bytes(workspace, "workspace", device)
    sv, sv_bytes = _bytes(saved, "saved", device)
    with _On(device, stream) as st:
        _check(_lib().ns_orthogonalize_stacks_backward(arr, len(grads), ctypes.byref(schedule.c), sv, sv_bytes, ws,
                                                       ws_bytes, st), "ns_orthogonalize_stacks_backward")


def orthogonalize_alloc(stacks: Sequence[Stack], schedule: Schedule, keep: bool = False):
    """ns_orthogonalize_stacks on torch's current stream with buffers of its own; returns the `saved`
    buffer if `keep`, else None."""
    arr, device = _stack_descs(stacks)
    lib, n, sch = _lib(), len(stacks), ctypes.byref(schedule.c)
    with _On(device, None) as st:
        ws = workspace(lib.ns_stacks_workspace_size(arr, n, sch, int(keep)), device=device)
        saved = workspace(lib.ns_stacks_saved_size(arr, n, sch), device=device) if keep else None
        _check(lib.ns_orthogonalize_stacks(arr, n, sch, saved.data_ptr() if keep else None, saved.numel() if keep else 0,
                                           ws.data_ptr(), ws.numel(), st), "ns_orthogonalize_stacks")
    return saved


def orthogonalize_backward_alloc(grads: Sequence[Stack], schedule: Schedule, saved):
    """ns_orthogonalize_stacks_backward on torch's current stream with a workspace of its own."""
    arr, device = _stack_descs(grads)
    lib, n, sch = _lib(), len(grads), ctypes.byref(schedule.c)
    with _On(device, None) as st:
        ws = workspace(lib.ns_stacks_backward_workspace_size(arr, n, sch), device=device)
        _check(lib.ns_orthogonalize_stacks_backward(arr, n, sch, saved.data_ptr(), saved.numel(), ws.data_ptr(), ws.numel(),
                                                    st), "ns_orthogonalize_stacks_backward")


def muon_stacks_workspace_size(stacks: Sequence[MuonStack], hp) -> int:
    return int(_lib().muon_stacks_workspace_size(_muon_stack_descs(stacks)[0], len(stacks), ctypes.byref(hp[0])))


def muon_step_stacks(stacks: Sequence[MuonStack], hp, workspace, grad_scale=None, stream=None):
    """The Muon step on every block of every stack; G is multiplied by the device scalar
    `grad_scale` first."""
    import torch
    arr, device = _muon_stack_descs(stacks)
    ws, ws_bytes = _bytes(workspace, "workspace", device)
    gs = _scalar(grad_scale, "grad_scale", device, torch.float32)
    with _On(device, stream) as st:
        _check(_lib().muon_step_stacks(arr, len(stacks), ctypes.byref(hp[0]), gs, ws, ws_bytes, st), "muon_step_stacks")


# ---------------------------------------------------------------------------- gradient norm, AdamW
# One row of 6 64-bit words per tensor, as adamw_tensor_desc lies in memory, made with maps over whole lists:
# sets of hundreds of small tensors cost more on the host than on the GPU otherwise.
def _adam_table(W, G, m, v, n, codes):
    table = array.array("q", itertools.chain.from_iterable(zip(W, G, m, v, n, codes)))
    return (AdamWTensorDesc * len(n)).from_buffer(table)


def _dense(tensors, name, device):
    """Checks that all are dense on `device`; returns their pointers and type codes."""
    import torch
    T = torch.Tensor
    codes = list(map(_codes().get, [t.dtype for t in tensors]))
    if not device.type == "cuda" or None in codes or not all(map(T.is_contiguous, tensors)) or \
            set(map(T.get_device, tensors)) != {device.index}:
        for t in tensors:      # one of them says what is wrong
            _need(t, name, device=device)
            _dtype16(t, name)
    return list(map(T.data_ptr, tensors)), codes


def _grad_descs(grads):
    import torch
    if not grads:
        raise ValueError("no gradients")
    device = grads[0].device
    ptrs, codes = _dense(grads, "G", device)
    none = itertools.repeat(0)
    return _adam_table(none, ptrs, none, none, list(map(torch.Tensor.numel, grads)), [c << 32 for c in codes]), device


def grad_norm_workspace_size(grads) -> int:
    return int(_lib().grad_norm_workspace_size(_grad_descs(grads)[0], len(grads)))


def grad_norm_batched(grads, max_norm: float, out, workspace, stream=None):
    """out[0] <- the norm of all gradients together, out[1] <- min(1, max_norm / (norm + 1e-6))."""
    import torch
    arr, device = _grad_descs(grads)
    _need(out, "out", device=device)
    if out.dtype != torch.float32 or out.numel() != 2:
        raise ValueError("out must hold two fp32 values")
    ws, ws_bytes = _bytes(workspace, "workspace", device)
    with _On(device, stream) as st:
        _check(_lib().grad_norm_batched(arr, len(grads), float(max_norm), out.data_ptr(), ws, ws_bytes, st),
               "grad_norm_batched")


def adamw_hyper(lr: float = 1e-3, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                weight_decay: float = 0.01) -> AdamWHyper:
    return AdamWHyper(float(lr), float(beta1), float(beta2), float(eps), float(weight_decay), 0, None)


def adamw_step_batched(tensors: Sequence[AdamWTensor], hp: AdamWHyper, step, grad_scale=None, stream=None):
    """AdamW on every tensor.  `step` is the number of this step, from 1: an int, or a device int64
    (read when the step runs, so that a captured step can be replayed as it advances)."""
    import torch
    if not tensors:
        raise ValueError("no tensors")
    W, G, m, v = [t.W for t in tensors], [t.G for t in tensors], [t.m for t in tensors], [t.v for t in tensors]
    shapes = [t.shape for t in W]
    if any([t.shape for t in x] != shapes for x in (G, m, v)):
        raise ValueError("W, G, m and v must have the same shape")
    device = W[0].device
    (wp, wc), (gp, gc), (mp, mc), (vp, vc) = (_dense(x, name, device) for x, name in
                                              ((W, "W"), (G, "G"), (m, "m"), (v, "v")))
    if {MUON_F32} != set(mc) | set(vc):
        raise TypeError("the moments m and v must be fp32")
    arr = _adam_table(wp, gp, mp, vp, list(map(torch.Tensor.numel, W)), [a | b << 32 for a, b in zip(wc, gc)])
    h = AdamWHyper(hp.lr, hp.beta1, hp.beta2, hp.eps, hp.weight_decay, 0, None)
    if isinstance(step, torch.Tensor):
        h.step_dev = _scalar(step, "step", device, torch.int64)
    else:
        h.step = int(step)
    gs = _scalar(grad_scale, "grad_scale", device, torch.float32)
    with _On(device, stream) as st:
        _check(_lib().adamw_step_batched(arr, len(tensors), ctypes.byref(h), gs, st), "adamw_step_batched")
