"""Python binding of the layer operators' C ABI (include/ptg_layer.h): the RMS norm with the residual's
addition, the product with bias, activation and residual in its epilogue, and their gradients.

Argument marshalling only, like the GEMM's binding. The function names are the C ABI's: layer_create,
layer_destroy, layer_sync, layer_last_hip_error, layer_rmsnorm, layer_rmsnorm_backward, layer_linear,
layer_activation_backward, layer_linear_backward. Matrices are 2-D device tensors whose rows are dense; the row
stride is free (a column slice of a wider buffer works). Streams are torch.cuda streams (default: the current
stream). Outputs are given by the caller.
"""

from __future__ import annotations

import ctypes
import struct

from . import GEMM_OK, PtgError, _stream_ptr, load_library

LAYER_F32, LAYER_BF16, LAYER_E4M3 = 0, 1, 2
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}

# exported names, in the order of the header
LAYER_ABI_FUNCTIONS = ("layer_create", "layer_destroy", "layer_sync", "layer_last_hip_error", "layer_rmsnorm",
                       "layer_rmsnorm_backward", "layer_linear", "layer_activation_backward", "layer_linear_backward")


def _struct(pointers, sizes, ints, floats=()):
    return ([(n, ctypes.c_void_p) for n in pointers] + [(n, ctypes.c_int64) for n in sizes] +
            [(n, ctypes.c_int32) for n in ints] + [(n, ctypes.c_float) for n in floats])


class RmsnormArgs(ctypes.Structure):
    _fields_ = _struct(("x", "residual", "weight", "sum_out", "out", "scale"), ("m", "n", "ldx", "ldr", "lds", "ldo"),
                       ("type", "weight_type", "out_type"), ("eps",))


class RmsnormGradArgs(ctypes.Structure):
    _fields_ = _struct(("dy", "s", "weight", "dsum", "dx", "dweight"), ("m", "n", "lddy", "lds", "lddsum", "lddx"),
                       ("type", "dy_type", "weight_type", "accumulate"), ("eps",))


class LinearArgs(ctypes.Structure):
    _fields_ = _struct(("x", "w", "x_scale", "w_scale", "bias", "residual", "pre", "out"),
                       ("m", "n", "k", "ldx", "ldw", "ldr", "ldp", "ldo"),
                       ("in_type", "bias_type", "residual_type", "out_type", "activation", "pad"))


class ActivationGradArgs(ctypes.Structure):
    _fields_ = _struct(("dout", "pre", "dpre", "dbias"), ("m", "n", "lddo", "ldp", "lddp"), ("activation", "accumulate"))


class LinearGradArgs(ctypes.Structure):
    _fields_ = _struct(("dpre", "x", "w", "dx", "dw"), ("m", "n", "k", "lddp", "ldx", "ldw", "lddx", "lddw"),
                       ("dx_type", "dw_type", "accumulate", "pad"))


def _packer(cls):
    """The structure's values as bytes in one call (setting ctypes fields one by one costs microseconds a call, which is
    what a decode step's small operators take on the device)."""
    codes = {ctypes.c_void_p: "P", ctypes.c_int64: "q", ctypes.c_int32: "i", ctypes.c_float: "f"}
    p = struct.Struct("@" + "".join(codes[t] for _, t in cls._fields_) + "0q")  # native sizes and alignment, padded to 8
    assert p.size == ctypes.sizeof(cls)
    return p.pack


_RMSNORM, _RMSNORM_GRAD, _LINEAR, _ACTIVATION_GRAD, _LINEAR_GRAD = (
    _packer(c) for c in (RmsnormArgs, RmsnormGradArgs, LinearArgs, ActivationGradArgs, LinearGradArgs))

_lib = None


def _library():
    global _lib
    if _lib is None:
        lib = load_library()
        vp = ctypes.c_void_p
        lib.layer_create.argtypes = [ctypes.POINTER(vp), ctypes.c_int32]
        lib.layer_destroy.argtypes = [vp]
        lib.layer_sync.argtypes = [vp]
        lib.layer_last_hip_error.argtypes = [vp]
        lib.layer_last_hip_error.restype = ctypes.c_char_p
        lib.layer_rmsnorm.argtypes = [vp, vp]
        lib.layer_rmsnorm_backward.argtypes = [vp, vp, vp]
        lib.layer_linear.argtypes = [vp, vp, vp]
        lib.layer_activation_backward.argtypes = [vp, vp, vp]
        lib.layer_linear_backward.argtypes = [vp, vp, vp]
        _lib = lib
    return _lib


def _check(status: int, what: str, plan=None) -> None:
    if status != GEMM_OK:
        lib = _library()
        detail = (lib.layer_last_hip_error(plan.handle) or b"").decode() if plan is not None and plan.handle else ""
        raise PtgError(status, what, detail or (lib.gemm_status_str(status) or b"").decode())


class LayerPlan:
    """A layer_cfg handle (owns the operators' scratch)."""

    def __init__(self, device: int = 0):
        self.handle = ctypes.c_void_p()
        self.device = int(device)
        _check(_library().layer_create(ctypes.byref(self.handle), self.device), "layer_create")

    def destroy(self) -> None:
        if self.handle:
            _library().layer_destroy(self.handle)
            self.handle = ctypes.c_void_p()

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.destroy()


def layer_create(device: int = 0) -> LayerPlan:
    """layer_create: a plan on `device` (the current device)."""
    return LayerPlan(device)


def layer_destroy(plan: LayerPlan) -> None:
    plan.destroy()


def layer_sync(plan: LayerPlan, strict: bool = True) -> int:
    """layer_sync: wait for the plan's last stream and return (strict=False) or raise on (strict=True) the
    device status of its products."""
    st = int(_library().layer_sync(plan.handle))
    if strict:
        _check(st, "layer_sync", plan)
    return st


def layer_last_hip_error(plan: LayerPlan) -> str:
    return (_library().layer_last_hip_error(plan.handle) or b"").decode()


_codes = {}      # torch dtype -> type code
_raw_stream = None  # device index -> the current stream's handle
_current_device = None


def _prepare():
    global _raw_stream, _current_device
    import torch
    _codes.update({torch.float32: LAYER_F32, torch.bfloat16: LAYER_BF16, torch.float8_e4m3fn: LAYER_E4M3})
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)
    _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _stream_of(stream, at):
    return _raw_stream(at) if stream is None else _stream_ptr(stream)


def _first(name, t, device=None):
    """(shape, device index) of the operand that the others are measured by; it is on `device` (a plan's) or the current
    one."""
    if not _codes:
        _prepare()
    at = t.get_device()
    if at < 0:
        raise ValueError(f"{name} must be a device tensor")
    if at != (_current_device() if device is None else device):
        raise ValueError(f"{name} is on {t.device}, the call's device is another one")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D")
    return shape, at


def _refuse(name, t, shape, at, allowed):
    """What is wrong with an argument that failed a check."""
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != at:
        raise ValueError(f"{name} is on {t.device}, expected device {at}")
    if _codes.get(t.dtype) not in allowed:
        raise ValueError(f"{name} has dtype {t.dtype}")
    raise ValueError(f"{name} must have dense rows (stride 1 along its columns)" if len(shape) == 2 else f"{name} must be contiguous")


def _matrix(name, t, shape, at, allowed):
    """(pointer, row stride, type code) of an optional matrix with dense rows."""
    if t is None:
        return 0, 0, LAYER_F32
    code = _codes.get(t.dtype)
    if t.shape != shape or t.get_device() != at or code not in allowed:
        _refuse(name, t, shape, at, allowed)
    rows, cols = shape
    if t.is_contiguous():
        return t.data_ptr(), cols, code
    row, col = t.stride()
    if col != 1 and cols > 1:
        _refuse(name, t, shape, at, allowed)
    return t.data_ptr(), row if rows > 1 else cols, code


def _vector(name, t, n, at, allowed):
    """(pointer, type code) of an optional dense vector of n elements."""
    if t is None:
        return 0, LAYER_F32
    code = _codes.get(t.dtype)
    if t.shape != (n,) or t.get_device() != at or code not in allowed or not t.is_contiguous():
        _refuse(name, t, (n,), at, allowed)
    return t.data_ptr(), code


def _activation(name) -> int:
    if name not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {list(ACTIVATIONS)}")
    return ACTIVATIONS[name]


_STREAM = (LAYER_F32, LAYER_BF16)
_ANY = (LAYER_F32, LAYER_BF16, LAYER_E4M3)
_ONLY = {c: (c,) for c in _ANY}  # the types allowed beside one that is given


def layer_rmsnorm(x, weight, out, *, residual=None, sum_out=None, scale=None, eps: float = 1e-6, stream=None) -> None:
    """layer_rmsnorm: out = s / sqrt(mean(s^2) + eps) * weight per row, s = x + residual (kept in sum_out, which
    may be x or residual). x, residual, sum_out: one dtype, bf16 or fp32. weight: bf16 or fp32, or None. out: fp32,
    bf16, or float8_e4m3fn with `scale` (fp32, one value a row): s's norm is then about out * scale[:, None]."""
    shape, at = _first("x", x)
    m, n = shape
    px, ldx, ty = _matrix("x", x, shape, at, _STREAM)
    pr, ldr, _ = _matrix("residual", residual, shape, at, _ONLY[ty])
    ps, lds, _ = _matrix("sum_out", sum_out, shape, at, _ONLY[ty])
    pw, wt = _vector("weight", weight, n, at, _STREAM)
    po, ldo, ot = _matrix("out", out, shape, at, _ANY)
    pc, _ = _vector("scale", scale, m, at, _ONLY[LAYER_F32])
    a = _RMSNORM(px, pr, pw, ps, po, pc, m, n, ldx, ldr, lds, ldo, ty, wt, ot, eps)
    st = (_lib or _library()).layer_rmsnorm(a, _stream_of(stream, at))
    if st:
        _check(st, "layer_rmsnorm")


def layer_rmsnorm_backward(dy, s, weight, dx, dweight, plan: LayerPlan, *, dsum=None, accumulate: bool = False,
                           eps: float = 1e-6, stream=None) -> None:
    """layer_rmsnorm_backward: dx (of the sum s, so of x and of the residual) and dweight (fp32) from dy, at s.
    dsum: the gradient that reaches s from elsewhere, added to dx (dx may be dsum). dx or dweight may be None."""
    shape, at = _first("s", s, plan.device)
    m, n = shape
    ps, lds, ty = _matrix("s", s, shape, at, _STREAM)
    pd, lddy, dt = _matrix("dy", dy, shape, at, _STREAM)
    pw, wt = _vector("weight", weight, n, at, _STREAM)
    pu, lddsum, _ = _matrix("dsum", dsum, shape, at, _ONLY[ty])
    px, lddx, _ = _matrix("dx", dx, shape, at, _ONLY[ty])
    pg, _ = _vector("dweight", dweight, n, at, _ONLY[LAYER_F32])
    a = _RMSNORM_GRAD(pd, ps, pw, pu, px, pg, m, n, lddy, lds, lddsum, lddx, ty, dt, wt, 1 if accumulate else 0, eps)
    st = (_lib or _library()).layer_rmsnorm_backward(a, plan.handle, _stream_of(stream, at))
    if st:
        _check(st, "layer_rmsnorm_backward", plan)


def layer_linear(x, w, out, plan: LayerPlan, *, bias=None, activation: str = "none", residual=None, pre=None, x_scale=None,
                 w_scale=None, stream=None) -> None:
    """layer_linear: out = act(x . w^T + bias) + residual, x: m x k, w: n x k, both bf16 or both float8_e4m3fn (then
    with row scales x_scale and w_scale, fp32). out and residual: bf16 or fp32; residual may be out. pre (bf16)
    keeps the activation's argument for layer_activation_backward."""
    act = _activation(activation)
    x_shape, at = _first("x", x, plan.device)
    w_shape, _ = _first("w", w, plan.device)
    m, k = x_shape
    n, k2 = w_shape
    if k2 != k:
        raise ValueError(f"shape mismatch: x {tuple(x.shape)}, w {tuple(w.shape)}")
    shape = (m, n)
    px, ldx, ty = _matrix("x", x, x_shape, at, (LAYER_BF16, LAYER_E4M3))
    pw, ldw, _ = _matrix("w", w, w_shape, at, _ONLY[ty])
    pxs, _ = _vector("x_scale", x_scale, m, at, _ONLY[LAYER_F32])
    pws, _ = _vector("w_scale", w_scale, n, at, _ONLY[LAYER_F32])
    pb, bt = _vector("bias", bias, n, at, _STREAM)
    pr, ldr, rt = _matrix("residual", residual, shape, at, _STREAM)
    pz, ldp, _ = _matrix("pre", pre, shape, at, _ONLY[LAYER_BF16])
    po, ldo, ot = _matrix("out", out, shape, at, _STREAM)
    a = _LINEAR(px, pw, pxs, pws, pb, pr, pz, po, m, n, k, ldx, ldw, ldr, ldp, ldo, ty, bt, rt, ot, act, 0)
    st = (_lib or _library()).layer_linear(a, plan.handle, _stream_of(stream, at))
    if st:
        _check(st, "layer_linear", plan)


def layer_activation_backward(dout, pre, dpre, plan: LayerPlan, *, activation: str = "none", dbias=None,
                              accumulate: bool = False, stream=None) -> None:
    """layer_activation_backward: dpre = dout * act'(pre) (bf16; dpre may be dout or pre, or None) and dbias = its
    column sums before rounding (fp32, or None). pre may be None with activation "none"."""
    act = _activation(activation)
    shape, at = _first("dout", dout, plan.device)
    m, n = shape
    pd, lddo, _ = _matrix("dout", dout, shape, at, _ONLY[LAYER_BF16])
    pz, ldp, _ = _matrix("pre", pre, shape, at, _ONLY[LAYER_BF16])
    pg, lddp, _ = _matrix("dpre", dpre, shape, at, _ONLY[LAYER_BF16])
    pb, _ = _vector("dbias", dbias, n, at, _ONLY[LAYER_F32])
    a = _ACTIVATION_GRAD(pd, pz, pg, pb, m, n, lddo, ldp, lddp, act, 1 if accumulate else 0)
    st = (_lib or _library()).layer_activation_backward(a, plan.handle, _stream_of(stream, at))
    if st:
        _check(st, "layer_activation_backward", plan)


def layer_linear_backward(dpre, x, w, plan: LayerPlan, *, dx=None, dw=None, accumulate: bool = False, stream=None) -> None:
    """layer_linear_backward: dx = dpre . w (m x k) and dw = dpre^T . x (n x k; added to dw with accumulate), each
    bf16 or fp32 and optional. dpre, x, w: bf16; x may be None without dw, w may be None without dx."""
    if (dx is None and dw is None) or (dx is not None and w is None) or (dw is not None and x is None):
        raise ValueError("layer_linear_backward needs dx or dw, w for dx and x for dw")
    shape, at = _first("dpre", dpre, plan.device)
    m, n = shape
    k = _first("w", w, plan.device)[0][1] if w is not None else _first("x", x, plan.device)[0][1]
    x_shape, w_shape = (m, k), (n, k)
    pd, lddp, _ = _matrix("dpre", dpre, shape, at, _ONLY[LAYER_BF16])
    px, ldx, _ = _matrix("x", x, x_shape, at, _ONLY[LAYER_BF16])
    pw, ldw, _ = _matrix("w", w, w_shape, at, _ONLY[LAYER_BF16])
    pdx, lddx, xt = _matrix("dx", dx, x_shape, at, _STREAM)
    pdw, lddw, wt = _matrix("dw", dw, w_shape, at, _STREAM)
    a = _LINEAR_GRAD(pd, px, pw, pdx, pdw, m, n, k, lddp, ldx, ldw, lddx, lddw, xt, wt, 1 if accumulate else 0, 0)
    st = (_lib or _library()).layer_linear_backward(a, plan.handle, _stream_of(stream, at))
    if st:
        _check(st, "layer_linear_backward", plan)
