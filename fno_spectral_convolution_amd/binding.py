"""ctypes binding of libfno (argument marshalling only).

Every function of ``include/fno.h`` and ``include/fno_train.h`` is exposed under its C name and
takes plain integers for pointers (``tensor.data_ptr()``) and streams
(``torch.cuda.current_stream().cuda_stream``).
``Plan`` wraps a plan for torch tensors: it allocates outputs, workspace and save buffers
with torch on the plan's device and forwards pointers; every step of the computation runs
in libfno's HIP kernels.  There is no fallback: if libfno.so is missing or fails to load,
importing this module raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
from ctypes import (POINTER, byref, c_char_p, c_double, c_float, c_int, c_int32, c_int64, c_size_t,
                    c_uint32, c_void_p)

_HERE = os.path.dirname(os.path.abspath(__file__))
# FNO_LIBRARY names another build of libfno (e.g. the host-sanitized one for CPU checks)
LIB_PATH = os.environ.get("FNO_LIBRARY") or os.path.join(_HERE, "libfno.so")

FNO_OK = 0
FNO_ERR_INVALID_ARGUMENT = 1
FNO_ERR_UNSUPPORTED = 2
FNO_ERR_HIP = 3
FNO_ERR_OUT_OF_MEMORY = 4
FNO_ERR_INTERNAL = 5

FNO_DTYPE_F32 = 0
FNO_DTYPE_BF16 = 1
FNO_DTYPE_F16 = 2

FNO_FLAG_TANH_PREACT = 1
FNO_FLAG_GELU = 2
FNO_FLAG_BIAS = 4
FNO_FLAG_INPUT_GELU = 8
FNO_FLAG_LAST_AXIS_FFT = 16
FNO_FLAG_LAST_AXIS_DENSE = 32

EXPORTS = [
    "fno_plan_validate", "fno_plan_create", "fno_plan_destroy", "fno_plan_query",
    "fno_plan_half_range", "fno_plan_last_axis_fft",
    "fno_spectral_conv_fwd", "fno_spectral_conv_bwd", "fno_block_fwd", "fno_block_fwd_static",
    "fno_block_bwd",
    "fno_block_fwd_mse", "fno_block_bwd_preact", "fno_pointwise_fwd", "fno_mse_workspace_bytes", "fno_mse_grad", "fno_mse_grad_scaled",
    "fno_tucker_order", "fno_tucker_create", "fno_tucker_destroy", "fno_tucker_query",
    "fno_tucker_keep_intermediates", "fno_tucker_save_bytes",
    "fno_tucker_block_fwd", "fno_tucker_block_bwd", "fno_tucker_spectral_conv_fwd",
    "fno_tucker_spectral_conv_bwd", "fno_tucker_block_fwd_mse", "fno_tucker_block_bwd_preact",
    "fno_timing_enable", "fno_timing_select",
    "fno_timing_reset", "fno_timing_count", "fno_timing_get", "fno_status_string",
    "fno_last_error_message",
]

# the training operators of fno_train.h
TRAIN_EXPORTS = [
    "fno_layer_norm_fwd", "fno_layer_norm_workspace_bytes", "fno_layer_norm_bwd",
    "fno_tensor_list_bytes", "fno_tensor_list_create", "fno_tensor_list_destroy",
    "fno_grad_norm_workspace_bytes", "fno_grad_norm", "fno_clip_grad_norm", "fno_adamw",
]


class fno_plan_desc(ctypes.Structure):
    _fields_ = [("ndim", c_int32), ("spectral_dtype", c_int32), ("flags", c_uint32),
                ("reserved", c_int32), ("batch", c_int64), ("c_in", c_int64),
                ("c_out", c_int64), ("n", c_int64 * 4), ("modes", c_int64 * 4)]


class fno_layer_norm_desc(ctypes.Structure):
    _fields_ = [("dtype", c_int32), ("reserved", c_int32), ("batch", c_int64),
                ("channels", c_int64), ("npts", c_int64), ("x_stride", c_int64),
                ("y_stride", c_int64), ("grad_x_stride", c_int64), ("eps", c_double)]


class fno_tensor(ctypes.Structure):
    _fields_ = [("data", c_void_p), ("elems", c_int64), ("dtype", c_int32),
                ("reserved", c_int32)]


class fno_adamw_desc(ctypes.Structure):
    _fields_ = [("lr", c_double), ("beta1", c_double), ("beta2", c_double), ("eps", c_double),
                ("weight_decay", c_double), ("step", c_int64)]


class FnoError(RuntimeError):
    def __init__(self, status: int, where: str, msg: str):
        super().__init__(f"{where}: {status_string(status)}: {msg}")
        self.status = status


def _load():
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libfno.so not built ({LIB_PATH}); run "
                           "`python -m fno_spectral_convolution_amd.build`")
    # torch brings its own HIP runtime; load it first so that libfno's libamdhip64
    # dependency resolves to that same, already loaded runtime (one HIP runtime per process:
    # libfno's kernels then run on torch's streams and memory).
    import torch  # noqa: F401
    lib = ctypes.CDLL(LIB_PATH)
    P = c_void_p
    sig = {
        "fno_plan_validate": (c_int, [POINTER(fno_plan_desc)]),
        "fno_plan_create": (c_int, [POINTER(fno_plan_desc), POINTER(c_void_p)]),
        "fno_plan_destroy": (c_int, [P]),
        "fno_plan_query": (c_int, [P, POINTER(c_size_t), POINTER(c_size_t), POINTER(c_size_t)]),
        "fno_plan_half_range": (c_int, [P, POINTER(c_int), c_int]),
        "fno_plan_last_axis_fft": (c_int, [P, POINTER(c_int)]),
        "fno_spectral_conv_fwd": (c_int, [P, P, P, P, P, P, c_size_t, P]),
        "fno_spectral_conv_bwd": (c_int, [P, P, P, P, P, P, P, P, c_size_t, P]),
        "fno_block_fwd": (c_int, [P, P, P, P, P, P, P, P, c_size_t, P]),
        "fno_block_fwd_static": (c_int, [P, P, P, P, P, P, P, P]),
        "fno_block_bwd": (c_int, [P, P, P, P, P, P, P, P, P, P, P, P, c_size_t, P]),
        "fno_block_fwd_mse": (c_int, [P, P, P, P, P, P, c_float, P, P, P, P, c_size_t, P]),
        "fno_block_bwd_preact": (c_int, [P, P, P, P, P, P, P, P, P, P, P, P, c_size_t, P]),
        "fno_pointwise_fwd": (c_int, [c_int64, c_int64, c_int64, c_int64, c_int64,
                                      P, P, P, P, P, P, P]),
        "fno_mse_workspace_bytes": (c_int, [c_int64, POINTER(c_size_t)]),
        "fno_mse_grad": (c_int, [c_int64, P, P, P, P, P, c_size_t, P]),
        "fno_mse_grad_scaled": (c_int, [c_int64, P, P, P, P, c_float, P, c_size_t, P]),
        "fno_tucker_order": (c_int, [POINTER(fno_plan_desc), POINTER(c_int32), c_char_p,
                                     c_size_t]),
        "fno_tucker_create": (c_int, [P, POINTER(c_int32), POINTER(c_void_p)]),
        "fno_tucker_destroy": (c_int, [P]),
        "fno_tucker_keep_intermediates": (c_int, [P, c_int]),
        "fno_tucker_save_bytes": (c_int, [P, POINTER(c_size_t)]),
        "fno_tucker_query": (c_int, [P, POINTER(c_size_t), POINTER(c_int64), POINTER(c_int64),
                                     c_char_p, c_size_t]),
        "fno_tucker_block_fwd": (c_int, [P, P, P, POINTER(c_void_p), P, P, P, P, P, c_size_t,
                                         P]),
        "fno_tucker_block_bwd": (c_int, [P, P, P, POINTER(c_void_p), P, P, P, P, P, P,
                                         POINTER(c_void_p), P, P, P, c_size_t, P]),
        "fno_tucker_spectral_conv_fwd": (c_int, [P, P, P, POINTER(c_void_p), P, P, P, c_size_t,
                                                 P]),
        "fno_tucker_spectral_conv_bwd": (c_int, [P, P, P, POINTER(c_void_p), P, P, P, P,
                                                 POINTER(c_void_p), P, c_size_t, P]),
        "fno_tucker_block_fwd_mse": (c_int, [P, P, P, POINTER(c_void_p), P, P, P, c_float, P,
                                             P, P, P, c_size_t, P]),
        "fno_tucker_block_bwd_preact": (c_int, [P, P, P, POINTER(c_void_p), P, P, P, P, P, P,
                                                POINTER(c_void_p), P, P, P, c_size_t, P]),
        "fno_layer_norm_fwd": (c_int, [POINTER(fno_layer_norm_desc), P, P, P, P, P, P]),
        "fno_layer_norm_workspace_bytes": (c_int, [POINTER(fno_layer_norm_desc),
                                                   POINTER(c_size_t)]),
        "fno_layer_norm_bwd": (c_int, [POINTER(fno_layer_norm_desc), P, P, P, P, P, P, P, P,
                                       c_size_t, P]),
        "fno_tensor_list_bytes": (c_int, [c_int64, P, POINTER(c_size_t)]),
        "fno_tensor_list_create": (c_int, [c_int64, P, P, c_size_t, P, POINTER(c_void_p)]),
        "fno_tensor_list_destroy": (c_int, [P]),
        "fno_grad_norm_workspace_bytes": (c_int, [P, POINTER(c_size_t)]),
        "fno_grad_norm": (c_int, [P, c_float, c_float, P, P, c_size_t, P]),
        "fno_clip_grad_norm": (c_int, [P, P, c_float, c_float, P, P, c_size_t, P]),
        "fno_adamw": (c_int, [P, P, P, P, POINTER(fno_adamw_desc), P, P]),
        "fno_timing_enable": (c_int, [c_int]),
        "fno_timing_select": (c_int, [c_char_p]),
        "fno_timing_reset": (c_int, []),
        "fno_timing_count": (c_int, [POINTER(c_int)]),
        "fno_timing_get": (c_int, [c_int, POINTER(c_char_p), POINTER(c_int64),
                                   POINTER(ctypes.c_double)]),
        "fno_status_string": (c_char_p, [c_int]),
        "fno_last_error_message": (c_char_p, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = _load()

import torch as _torch  # noqa: E402  (after libfno: _load has imported it)


def status_string(status: int) -> str:
    return _lib.fno_status_string(status).decode()


def last_error_message() -> str:
    return _lib.fno_last_error_message().decode()


def _check(status: int, where: str):
    if status != FNO_OK:
        raise FnoError(status, where, last_error_message())


def make_desc(batch, c_in, c_out, grid, modes, dtype=FNO_DTYPE_F32, flags=0) -> fno_plan_desc:
    d = fno_plan_desc()
    d.ndim = len(grid)
    d.spectral_dtype = dtype
    d.flags = flags
    d.reserved = 0
    d.batch, d.c_in, d.c_out = batch, c_in, c_out
    for j in range(4):
        d.n[j] = grid[j] if j < len(grid) else 0
        d.modes[j] = modes[j] if j < len(modes) else 0
    return d


# ---- raw C entry points (same names as the header) ----------------------------------------
def fno_plan_validate(desc: fno_plan_desc) -> int:
    return _lib.fno_plan_validate(byref(desc))


def fno_plan_create(desc: fno_plan_desc) -> int:
    out = c_void_p()
    _check(_lib.fno_plan_create(byref(desc), byref(out)), "fno_plan_create")
    return out.value


def fno_plan_destroy(plan: int) -> None:
    _check(_lib.fno_plan_destroy(plan), "fno_plan_destroy")


def fno_plan_query(plan: int):
    ws, sv, we = c_size_t(), c_size_t(), c_size_t()
    _check(_lib.fno_plan_query(plan, byref(ws), byref(sv), byref(we)), "fno_plan_query")
    return ws.value, sv.value, we.value


def fno_plan_half_range(plan: int, clear: bool = False) -> bool:
    """Whether a call on this IEEE-half plan wrote a non-finite output (synchronous read)."""
    v = c_int()
    _check(_lib.fno_plan_half_range(plan, byref(v), int(bool(clear))), "fno_plan_half_range")
    return bool(v.value)


def fno_plan_last_axis_fft(plan: int) -> bool:
    """Whether the plan takes its contiguous-axis forward transform by FFT (host only)."""
    v = c_int()
    _check(_lib.fno_plan_last_axis_fft(plan, byref(v)), "fno_plan_last_axis_fft")
    return bool(v.value)


def fno_spectral_conv_fwd(plan, x, w, y_spec, save, ws, ws_bytes, stream):
    _check(_lib.fno_spectral_conv_fwd(plan, x, w, y_spec, save, ws, ws_bytes, stream),
           "fno_spectral_conv_fwd")


def fno_spectral_conv_bwd(plan, x, w, save, grad_y_spec, grad_x, grad_w, ws, ws_bytes, stream):
    _check(_lib.fno_spectral_conv_bwd(plan, x, w, save, grad_y_spec, grad_x, grad_w, ws,
                                      ws_bytes, stream), "fno_spectral_conv_bwd")


def fno_block_fwd(plan, x, w, w_bypass, bias, y, save, ws, ws_bytes, stream):
    _check(_lib.fno_block_fwd(plan, x, w, w_bypass, bias, y, save, ws, ws_bytes, stream),
           "fno_block_fwd")


def fno_block_fwd_static(plan, x, w, w_bypass, bias, y, save, stream):
    _check(_lib.fno_block_fwd_static(plan, x, w, w_bypass, bias, y, save, stream),
           "fno_block_fwd_static")


def fno_block_bwd(plan, x, w, w_bypass, bias, save, grad_y, grad_x, grad_w, grad_w_bypass,
                  grad_bias, ws, ws_bytes, stream):
    _check(_lib.fno_block_bwd(plan, x, w, w_bypass, bias, save, grad_y, grad_x, grad_w,
                              grad_w_bypass, grad_bias, ws, ws_bytes, stream), "fno_block_bwd")


def fno_block_fwd_mse(plan, x, w, w_bypass, bias, target, grad_scale, grad_z, loss, save, ws,
                      ws_bytes, stream):
    _check(_lib.fno_block_fwd_mse(plan, x, w, w_bypass, bias, target, grad_scale, grad_z, loss,
                                  save, ws, ws_bytes, stream), "fno_block_fwd_mse")


def fno_block_bwd_preact(plan, x, w, w_bypass, bias, save, grad_z, grad_x, grad_w,
                         grad_w_bypass, grad_bias, ws, ws_bytes, stream):
    _check(_lib.fno_block_bwd_preact(plan, x, w, w_bypass, bias, save, grad_z, grad_x, grad_w,
                                     grad_w_bypass, grad_bias, ws, ws_bytes, stream),
           "fno_block_bwd_preact")


def fno_pointwise_fwd(batch, npts, c_in, hidden, c_out, x, w1, b1, w2, b2, y, stream):
    _check(_lib.fno_pointwise_fwd(batch, npts, c_in, hidden, c_out, x, w1, b1, w2, b2, y,
                                  stream), "fno_pointwise_fwd")


def fno_mse_workspace_bytes(n: int) -> int:
    b = c_size_t()
    _check(_lib.fno_mse_workspace_bytes(n, byref(b)), "fno_mse_workspace_bytes")
    return b.value


def fno_mse_grad(n, y, t, grad, loss, ws, ws_bytes, stream):
    _check(_lib.fno_mse_grad(n, y, t, grad, loss, ws, ws_bytes, stream), "fno_mse_grad")


def fno_mse_grad_scaled(n, y, t, grad, loss, grad_scale, ws, ws_bytes, stream):
    _check(_lib.fno_mse_grad_scaled(n, y, t, grad, loss, grad_scale, ws, ws_bytes, stream),
           "fno_mse_grad_scaled")


def fno_layer_norm_fwd(desc, x, gamma, beta, y, stats, stream):
    _check(_lib.fno_layer_norm_fwd(byref(desc), x, gamma, beta, y, stats, stream),
           "fno_layer_norm_fwd")


def fno_layer_norm_workspace_bytes(desc) -> int:
    b = c_size_t()
    _check(_lib.fno_layer_norm_workspace_bytes(byref(desc), byref(b)),
           "fno_layer_norm_workspace_bytes")
    return b.value


def fno_layer_norm_bwd(desc, x, gamma, stats, grad_y, grad_x, grad_gamma, grad_beta, ws, ws_bytes,
                       stream):
    _check(_lib.fno_layer_norm_bwd(byref(desc), x, gamma, stats, grad_y, grad_x, grad_gamma,
                                   grad_beta, ws, ws_bytes, stream), "fno_layer_norm_bwd")


def fno_tensor_list_bytes(count, tensors) -> int:
    b = c_size_t()
    _check(_lib.fno_tensor_list_bytes(count, tensors, byref(b)), "fno_tensor_list_bytes")
    return b.value


def fno_tensor_list_create(count, tensors, table, table_bytes, stream) -> int:
    out = c_void_p()
    _check(_lib.fno_tensor_list_create(count, tensors, table, table_bytes, stream, byref(out)),
           "fno_tensor_list_create")
    return out.value


def fno_tensor_list_destroy(handle) -> None:
    _check(_lib.fno_tensor_list_destroy(handle), "fno_tensor_list_destroy")


def fno_grad_norm_workspace_bytes(grads) -> int:
    b = c_size_t()
    _check(_lib.fno_grad_norm_workspace_bytes(grads, byref(b)), "fno_grad_norm_workspace_bytes")
    return b.value


def fno_grad_norm(grads, max_norm, grad_scale, record, ws, ws_bytes, stream):
    _check(_lib.fno_grad_norm(grads, max_norm, grad_scale, record, ws, ws_bytes, stream),
           "fno_grad_norm")


def fno_clip_grad_norm(grads, out, max_norm, grad_scale, record, ws, ws_bytes, stream):
    _check(_lib.fno_clip_grad_norm(grads, out, max_norm, grad_scale, record, ws, ws_bytes,
                                   stream), "fno_clip_grad_norm")


def fno_adamw(params, grads, exp_avg, exp_avg_sq, desc, record, stream):
    _check(_lib.fno_adamw(params, grads, exp_avg, exp_avg_sq, byref(desc), record, stream),
           "fno_adamw")


def fno_timing_enable(enable: bool) -> None:
    _check(_lib.fno_timing_enable(1 if enable else 0), "fno_timing_enable")


def fno_timing_select(name=None) -> None:
    """Time only the launches of kernel `name` (None: every launch)."""
    _check(_lib.fno_timing_select(name.encode() if name else None), "fno_timing_select")


def fno_timing_reset() -> None:
    _check(_lib.fno_timing_reset(), "fno_timing_reset")


def fno_timing_count() -> int:
    n = c_int()
    _check(_lib.fno_timing_count(byref(n)), "fno_timing_count")
    return n.value


def fno_timing_get(index: int):
    name, launches, ms = c_char_p(), c_int64(), ctypes.c_double()
    _check(_lib.fno_timing_get(index, byref(name), byref(launches), byref(ms)), "fno_timing_get")
    return name.value.decode(), launches.value, ms.value


def timing_report() -> dict:
    """{kernel name: (launches, total ms)} of everything recorded since the last reset."""
    return {nm: (n, ms) for nm, n, ms in (fno_timing_get(i) for i in range(fno_timing_count()))}


# ---- torch-facing convenience (allocation + pointer marshalling only) ---------------------
def spectral_dtype(mixed):
    """fno_dtype of a plan: False -> F32, True / "bf16" -> BF16, "f16" -> F16."""
    if mixed is False or mixed is None:
        return FNO_DTYPE_F32
    if mixed is True or mixed == "bf16":
        return FNO_DTYPE_BF16
    if mixed == "f16":
        return FNO_DTYPE_F16
    raise ValueError(f"unknown spectral precision {mixed!r}")


def _ptr(t):
    return None if t is None else t.data_ptr()


class Plan:
    """One FNO block shape.  Tensors are torch tensors on the plan's device: fields float32
    [B, C, *grid], spectral weights complex64 [2^(d-1), Cin, Cout, *modes], bypass float32
    [Cout, Cin], bias float32 [Cout]."""

    def __init__(self, batch, c_in, c_out, grid, modes, mixed=False, tanh=None, gelu=True,
                 bias=True, device=None, input_gelu=False, last_axis=None):
        """mixed: False (fp32 spectral path), True or "bf16" (bfloat16 operands), "f16" (IEEE
        half operands); a mixed plan takes the tanh pre-activation unless tanh says otherwise.
        input_gelu: x is a pre-activation and the block's input is GELU(x).
        last_axis: None (the plan picks), "fft" or "dense": how a float32 plan takes the
        forward transform of the contiguous axis."""
        import torch
        self.torch = torch
        self.device = torch.device(device) if device is not None else torch.device("cuda")
        tanh = bool(mixed) if tanh is None else tanh
        flags = (FNO_FLAG_TANH_PREACT if tanh else 0) | (FNO_FLAG_GELU if gelu else 0) | \
            (FNO_FLAG_BIAS if bias else 0) | (FNO_FLAG_INPUT_GELU if input_gelu else 0)
        if last_axis not in (None, "fft", "dense"):
            raise ValueError(f"last_axis must be None, 'fft' or 'dense', not {last_axis!r}")
        flags |= {None: 0, "fft": FNO_FLAG_LAST_AXIS_FFT,
                  "dense": FNO_FLAG_LAST_AXIS_DENSE}[last_axis]
        self.desc = make_desc(batch, c_in, c_out, tuple(grid), tuple(modes),
                              spectral_dtype(mixed), flags)
        self.batch, self.c_in, self.c_out = batch, c_in, c_out
        self.grid, self.modes = tuple(grid), tuple(modes)
        self.flags = flags
        with torch.cuda.device(self.device):
            self.handle = fno_plan_create(self.desc)
        self.ws_bytes, self.save_bytes, self.weight_elems = fno_plan_query(self.handle)
        self._ws = None

    def close(self):
        if getattr(self, "handle", None):
            fno_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def half_range_exceeded(self, clear=False):
        """IEEE-half plans: whether a call since creation (or the last clear) wrote a
        non-finite output; synchronise the calls' streams first."""
        return fno_plan_half_range(self.handle, clear)

    @property
    def last_axis_fft(self):
        """True when the plan takes its contiguous-axis forward transform by FFT."""
        return fno_plan_last_axis_fft(self.handle)

    # buffers
    def workspace(self):
        if self._ws is None:
            self._ws = self.torch.empty(max(self.ws_bytes, 16), dtype=self.torch.uint8,
                                        device=self.device)
        return self._ws

    def new_save(self):
        return self.torch.empty(max(self.save_bytes, 16), dtype=self.torch.uint8,
                                device=self.device)

    def _field(self, c):
        return self.torch.empty((self.batch, c) + self.grid, dtype=self.torch.float32,
                                device=self.device)

    def _stream(self):
        return self.torch.cuda.current_stream(self.device).cuda_stream

    # entry points
    def spectral_conv_fwd(self, x, w, save=None, out=None):
        y = out if out is not None else self._field(self.c_out)
        ws = self.workspace()
        fno_spectral_conv_fwd(self.handle, x.data_ptr(), w.data_ptr(), y.data_ptr(), _ptr(save),
                              ws.data_ptr(), self.ws_bytes, self._stream())
        return y

    def spectral_conv_bwd(self, x, w, grad_y_spec, save=None, want_x=True, want_w=True):
        gx = self._field(self.c_in) if want_x else None
        gw = self.torch.empty_like(w) if want_w else None
        ws = self.workspace()
        fno_spectral_conv_bwd(self.handle, x.data_ptr(), w.data_ptr(), _ptr(save),
                              grad_y_spec.data_ptr(), _ptr(gx), _ptr(gw), ws.data_ptr(),
                              self.ws_bytes, self._stream())
        return gx, gw

    def block_fwd(self, x, w, wb, bias=None, save=None, out=None):
        y = out if out is not None else self._field(self.c_out)
        ws = self.workspace()
        fno_block_fwd(self.handle, x.data_ptr(), w.data_ptr(), wb.data_ptr(), _ptr(bias),
                      y.data_ptr(), _ptr(save), ws.data_ptr(), self.ws_bytes, self._stream())
        return y

    def block_fwd_static(self, x, w, wb, bias=None, save=None, out=None):
        """block_fwd on libfno's static scratch (no workspace is allocated for it)."""
        y = out if out is not None else self._field(self.c_out)
        fno_block_fwd_static(self.handle, x.data_ptr(), w.data_ptr(), wb.data_ptr(), _ptr(bias),
                             y.data_ptr(), _ptr(save), self._stream())
        return y

    def block_bwd(self, x, w, wb, bias, save, grad_y, want=("x", "w", "wb", "bias"), out=None):
        t = self.torch
        o = out or {}
        # an output is allocated only when the caller passes none for it
        gx = o["x"] if "x" in o else (self._field(self.c_in) if "x" in want else None)
        gw = o["w"] if "w" in o else (t.empty_like(w) if "w" in want else None)
        gwb = o["wb"] if "wb" in o else (t.empty_like(wb) if "wb" in want else None)
        gb = o["bias"] if "bias" in o else (
            t.empty(self.c_out, dtype=t.float32, device=self.device) if "bias" in want
            else None)
        ws = self.workspace()
        fno_block_bwd(self.handle, x.data_ptr(), w.data_ptr(), wb.data_ptr(), _ptr(bias),
                      _ptr(save), grad_y.data_ptr(), _ptr(gx), _ptr(gw), _ptr(gwb), _ptr(gb),
                      ws.data_ptr(), self.ws_bytes, self._stream())
        return {"x": gx, "w": gw, "wb": gwb, "bias": gb}

    def block_fwd_mse(self, x, w, wb, bias, target, grad_scale=1.0, save=None, grad_z=None,
                      loss=None):
        """Block forward fused with the MSE loss; returns (grad_z, loss) (device tensors)."""
        t = self.torch
        gz = grad_z if grad_z is not None else self._field(self.c_out)
        ls = loss if loss is not None else t.empty(1, dtype=t.float32, device=self.device)
        ws = self.workspace()
        fno_block_fwd_mse(self.handle, x.data_ptr(), w.data_ptr(), wb.data_ptr(), _ptr(bias),
                          target.data_ptr(), float(grad_scale), gz.data_ptr(), ls.data_ptr(),
                          _ptr(save), ws.data_ptr(), self.ws_bytes, self._stream())
        return gz, ls

    def block_bwd_preact(self, x, w, wb, bias, save, grad_z, want=("x", "w", "wb", "bias"),
                         out=None):
        """Block backward from the gradient at the pre-activation (block_bwd's outputs)."""
        t = self.torch
        o = out or {}
        # an output is allocated only when the caller passes none for it
        gx = o["x"] if "x" in o else (self._field(self.c_in) if "x" in want else None)
        gw = o["w"] if "w" in o else (t.empty_like(w) if "w" in want else None)
        gwb = o["wb"] if "wb" in o else (t.empty_like(wb) if "wb" in want else None)
        gb = o["bias"] if "bias" in o else (
            t.empty(self.c_out, dtype=t.float32, device=self.device) if "bias" in want
            else None)
        ws = self.workspace()
        fno_block_bwd_preact(self.handle, x.data_ptr(), w.data_ptr(), wb.data_ptr(), _ptr(bias),
                             _ptr(save), grad_z.data_ptr(), _ptr(gx), _ptr(gw), _ptr(gwb),
                             _ptr(gb), ws.data_ptr(), self.ws_bytes, self._stream())
        return {"x": gx, "w": gw, "wb": gwb, "bias": gb}


def _ranks_arr(ranks):
    return (c_int32 * len(ranks))(*[int(r) for r in ranks])


def _ptr_arr(ptrs):
    return (c_void_p * len(ptrs))(*[p if p else None for p in ptrs])


def fno_tucker_order(desc, ranks) -> str:
    """The greedy contraction order of a descriptor and Tucker ranks (host only)."""
    buf = ctypes.create_string_buffer(512)
    _check(_lib.fno_tucker_order(byref(desc), _ranks_arr(ranks), buf, len(buf)),
           "fno_tucker_order")
    return buf.value.decode()


def fno_tucker_create(plan_handle, ranks):
    h = c_void_p()
    _check(_lib.fno_tucker_create(plan_handle, _ranks_arr(ranks), byref(h)), "fno_tucker_create")
    return h.value


def fno_tucker_destroy(handle):
    _check(_lib.fno_tucker_destroy(handle), "fno_tucker_destroy")


def fno_tucker_query(handle, nfactors):
    ws = c_size_t()
    core = c_int64()
    fac = (c_int64 * nfactors)()
    buf = ctypes.create_string_buffer(512)
    _check(_lib.fno_tucker_query(handle, byref(ws), byref(core), fac, buf, len(buf)),
           "fno_tucker_query")
    return ws.value, core.value, list(fac), buf.value.decode()


def fno_tucker_block_fwd(h, x, core, factors, wb, bias, y, save, ws, ws_bytes, stream):
    _check(_lib.fno_tucker_block_fwd(h, x, core, _ptr_arr(factors), wb, bias, y, save, ws,
                                     ws_bytes, stream), "fno_tucker_block_fwd")


def fno_tucker_block_bwd(h, x, core, factors, wb, bias, save, gy, gx, gcore, gfactors, gwb, gb,
                         ws, ws_bytes, stream):
    gf = _ptr_arr(gfactors) if gfactors is not None else None
    _check(_lib.fno_tucker_block_bwd(h, x, core, _ptr_arr(factors), wb, bias, save, gy, gx,
                                     gcore, gf, gwb, gb, ws, ws_bytes, stream),
           "fno_tucker_block_bwd")


def fno_tucker_block_fwd_mse(h, x, core, factors, wb, bias, target, grad_scale, grad_z, loss,
                             save, ws, ws_bytes, stream):
    _check(_lib.fno_tucker_block_fwd_mse(h, x, core, _ptr_arr(factors), wb, bias, target,
                                         grad_scale, grad_z, loss, save, ws, ws_bytes, stream),
           "fno_tucker_block_fwd_mse")


def fno_tucker_block_bwd_preact(h, x, core, factors, wb, bias, save, gz, gx, gcore, gfactors,
                                gwb, gb, ws, ws_bytes, stream):
    gf = _ptr_arr(gfactors) if gfactors is not None else None
    _check(_lib.fno_tucker_block_bwd_preact(h, x, core, _ptr_arr(factors), wb, bias, save, gz,
                                            gx, gcore, gf, gwb, gb, ws, ws_bytes, stream),
           "fno_tucker_block_bwd_preact")


def fno_tucker_spectral_conv_fwd(h, x, core, factors, y, save, ws, ws_bytes, stream):
    _check(_lib.fno_tucker_spectral_conv_fwd(h, x, core, _ptr_arr(factors), y, save, ws,
                                             ws_bytes, stream), "fno_tucker_spectral_conv_fwd")


def fno_tucker_spectral_conv_bwd(h, x, core, factors, save, gys, gx, gcore, gfactors, ws,
                                 ws_bytes, stream):
    gf = _ptr_arr(gfactors) if gfactors is not None else None
    _check(_lib.fno_tucker_spectral_conv_bwd(h, x, core, _ptr_arr(factors), save, gys, gx, gcore,
                                             gf, ws, ws_bytes, stream),
           "fno_tucker_spectral_conv_bwd")


class Tucker:
    """Tucker-factorised spectral weights bound to a ``Plan``: core complex64
    [R_in, R_out, R_0, .., R_{d-1}], factors complex64 [C_in, R_in], [C_out, R_out],
    [2 m_j, R_j] (outer axes), [m_{d-1}, R_{d-1}]."""

    def __init__(self, plan, ranks):
        self.plan = plan
        self.ranks = tuple(int(r) for r in ranks)
        self.nf = len(plan.grid) + 2
        if len(self.ranks) != self.nf:
            raise ValueError(f"need {self.nf} ranks (in, out, one per axis)")
        self.handle = fno_tucker_create(plan.handle, self.ranks)
        self.ws_bytes, self.core_elems, self.factor_elems, self.order = \
            fno_tucker_query(self.handle, self.nf)
        self._ws = None

    def close(self):
        if getattr(self, "handle", None):
            fno_tucker_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def factor_shapes(self):
        p = self.plan
        full = [p.c_in, p.c_out] + [2 * m for m in p.modes[:-1]] + [p.modes[-1]]
        return [(n, r) for n, r in zip(full, self.ranks)]

    def workspace(self):
        if self._ws is None:
            t = self.plan.torch
            self._ws = t.empty(max(self.ws_bytes, 16), dtype=t.uint8, device=self.plan.device)
        return self._ws

    def keep_intermediates(self, keep=True):
        """Keep the forward's weight-step intermediates in the save buffer for the backward
        (save buffers then come from new_save())."""
        _check(_lib.fno_tucker_keep_intermediates(self.handle, 1 if keep else 0),
               "fno_tucker_keep_intermediates")

    @property
    def save_bytes(self):
        b = c_size_t()
        _check(_lib.fno_tucker_save_bytes(self.handle, byref(b)), "fno_tucker_save_bytes")
        return b.value

    def new_save(self):
        t = self.plan.torch
        return t.empty(max(self.save_bytes, 16), dtype=t.uint8, device=self.plan.device)

    def block_fwd(self, x, core, factors, wb, bias=None, save=None, out=None):
        p = self.plan
        y = out if out is not None else p._field(p.c_out)
        ws = self.workspace()
        fno_tucker_block_fwd(self.handle, x.data_ptr(), core.data_ptr(),
                             [f.data_ptr() for f in factors], wb.data_ptr(), _ptr(bias),
                             y.data_ptr(), _ptr(save), ws.data_ptr(), self.ws_bytes,
                             p._stream())
        return y

    def spectral_conv_fwd(self, x, core, factors, save=None, out=None):
        p = self.plan
        y = out if out is not None else p._field(p.c_out)
        ws = self.workspace()
        fno_tucker_spectral_conv_fwd(self.handle, x.data_ptr(), core.data_ptr(),
                                     [f.data_ptr() for f in factors], y.data_ptr(), _ptr(save),
                                     ws.data_ptr(), self.ws_bytes, p._stream())
        return y

    def spectral_conv_bwd(self, x, core, factors, grad_y_spec, save=None, want_x=True,
                          want_w=True):
        """Returns (grad_x, grad_core, grad_factors) (None where not asked)."""
        p = self.plan
        t = p.torch
        gx = p._field(p.c_in) if want_x else None
        gcore = t.empty_like(core) if want_w else None
        gfac = [t.empty_like(f) for f in factors] if want_w else None
        ws = self.workspace()
        fno_tucker_spectral_conv_bwd(self.handle, x.data_ptr(), core.data_ptr(),
                                     [f.data_ptr() for f in factors], _ptr(save),
                                     grad_y_spec.data_ptr(), _ptr(gx), _ptr(gcore),
                                     [_ptr(g) for g in gfac] if gfac is not None else None,
                                     ws.data_ptr(), self.ws_bytes, p._stream())
        return gx, gcore, gfac

    def block_bwd(self, x, core, factors, wb, bias, save, grad_y, want_x=True, want_w=True,
                  out=None):
        """Returns dict(x, core, factors, wb, bias) of gradients (None where not asked)."""
        p = self.plan
        t = p.torch
        o = out or {}
        # an output is allocated only when the caller passes none for it
        gx = o["x"] if "x" in o else (p._field(p.c_in) if want_x else None)
        gcore = o["core"] if "core" in o else (t.empty_like(core) if want_w else None)
        gfac = o["factors"] if "factors" in o else (
            [t.empty_like(f) for f in factors] if want_w else None)
        gwb = o["wb"] if "wb" in o else t.empty_like(wb)
        gb = o["bias"] if "bias" in o else t.empty(p.c_out, dtype=t.float32, device=p.device)
        ws = self.workspace()
        fno_tucker_block_bwd(self.handle, x.data_ptr(), core.data_ptr(),
                             [f.data_ptr() for f in factors], wb.data_ptr(), _ptr(bias),
                             _ptr(save), grad_y.data_ptr(), _ptr(gx), _ptr(gcore),
                             [_ptr(g) for g in gfac] if gfac is not None else None,
                             _ptr(gwb), _ptr(gb), ws.data_ptr(), self.ws_bytes, p._stream())
        return {"x": gx, "core": gcore, "factors": gfac, "wb": gwb, "bias": gb}

    def block_fwd_mse(self, x, core, factors, wb, bias, target, grad_scale=1.0, save=None,
                      grad_z=None, loss=None):
        """block_fwd fused with the MSE loss; returns (grad_z, loss) (device tensors)."""
        p = self.plan
        t = p.torch
        gz = grad_z if grad_z is not None else p._field(p.c_out)
        ls = loss if loss is not None else t.empty(1, dtype=t.float32, device=p.device)
        ws = self.workspace()
        fno_tucker_block_fwd_mse(self.handle, x.data_ptr(), core.data_ptr(),
                                 [f.data_ptr() for f in factors], wb.data_ptr(), _ptr(bias),
                                 target.data_ptr(), float(grad_scale), gz.data_ptr(),
                                 ls.data_ptr(), _ptr(save), ws.data_ptr(), self.ws_bytes,
                                 p._stream())
        return gz, ls

    def block_bwd_preact(self, x, core, factors, wb, bias, save, grad_z, want_x=True,
                         want_w=True, out=None):
        """block_bwd from the gradient at the pre-activation (block_bwd's outputs)."""
        p = self.plan
        t = p.torch
        o = out or {}
        # an output is allocated only when the caller passes none for it
        gx = o["x"] if "x" in o else (p._field(p.c_in) if want_x else None)
        gcore = o["core"] if "core" in o else (t.empty_like(core) if want_w else None)
        gfac = o["factors"] if "factors" in o else (
            [t.empty_like(f) for f in factors] if want_w else None)
        gwb = o["wb"] if "wb" in o else t.empty_like(wb)
        gb = o["bias"] if "bias" in o else t.empty(p.c_out, dtype=t.float32, device=p.device)
        ws = self.workspace()
        fno_tucker_block_bwd_preact(self.handle, x.data_ptr(), core.data_ptr(),
                                    [f.data_ptr() for f in factors], wb.data_ptr(), _ptr(bias),
                                    _ptr(save), grad_z.data_ptr(), _ptr(gx), _ptr(gcore),
                                    [_ptr(g) for g in gfac] if gfac is not None else None,
                                    _ptr(gwb), _ptr(gb), ws.data_ptr(), self.ws_bytes,
                                    p._stream())
        return {"x": gx, "core": gcore, "factors": gfac, "wb": gwb, "bias": gb}


def pointwise(x, w1, b1=None, w2=None, b2=None, out=None):
    """Lift (w2 None) or projection head on a torch field [B, Cin, *grid]."""
    import torch
    batch, cin = x.shape[0], x.shape[1]
    npts = x[0, 0].numel()
    hidden = 0 if w2 is None else w1.shape[0]
    cout = w1.shape[0] if w2 is None else w2.shape[0]
    y = out if out is not None else torch.empty((batch, cout) + tuple(x.shape[2:]),
                                                dtype=torch.float32, device=x.device)
    fno_pointwise_fwd(batch, npts, cin, hidden, cout, x.data_ptr(), w1.data_ptr(), _ptr(b1),
                      _ptr(w2), _ptr(b2), y.data_ptr(),
                      torch.cuda.current_stream(x.device).cuda_stream)
    return y


def mse_grad(y, t, grad=None, loss=None, ws=None, grad_scale=1.0):
    """loss = mean((y - t)^2), grad = grad_scale * 2 (y - t) / n (grad_scale: a static loss
    scale for IEEE-half plans)."""
    import torch
    n = y.numel()
    g = grad if grad is not None else torch.empty_like(y)
    lo = loss if loss is not None else torch.empty(1, dtype=torch.float32, device=y.device)
    nb = fno_mse_workspace_bytes(n)
    w = ws if ws is not None else torch.empty(max(nb, 16), dtype=torch.uint8, device=y.device)
    stream = torch.cuda.current_stream(y.device).cuda_stream
    if grad_scale == 1.0:
        fno_mse_grad(n, y.data_ptr(), t.data_ptr(), g.data_ptr(), lo.data_ptr(), w.data_ptr(),
                     w.numel(), stream)
    else:
        fno_mse_grad_scaled(n, y.data_ptr(), t.data_ptr(), g.data_ptr(), lo.data_ptr(),
                            float(grad_scale), w.data_ptr(), w.numel(), stream)
    return lo, g


# ---- training operators -----------------------------------------------------------------------
# These are small next to a launch, so their argument checks are kept cheap: one dictionary, one
# attribute or one comparison each.
_KINDS = {_torch.float32: FNO_DTYPE_F32, _torch.bfloat16: FNO_DTYPE_BF16,
          _torch.float16: FNO_DTYPE_F16}
_LIST_KINDS = {**_KINDS, _torch.complex64: FNO_DTYPE_F32}  # as pairs of float32


# The handle of a device's current stream and the current device, without the Stream object and the
# set-up check of the public calls (0.1 us each against 1.9 and 0.3, next to 3.3 for a launch); the
# public calls where torch has no such functions.
_stream_handle = getattr(_torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: _torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(_torch._C, "_cuda_getDevice", None) or _torch.cuda.current_device


def _on_stream(index, fn, *args):
    """fn(*args, current stream of device `index`), with that device current."""
    if index == _current_device():
        return fn(*args, _stream_handle(index))
    with _torch.cuda.device(index):
        return fn(*args, _stream_handle(index))


def _vector(t, shape, index, name):
    """The address of packed float32 values of a shape on device `index` (None: none given)."""
    if t is None:
        return None
    if t.dtype != _torch.float32 or t.shape != shape or t.get_device() != index \
            or not t.is_contiguous():
        raise ValueError(f"{name}: needs packed float32 {tuple(shape)} on cuda:{index}")
    return t.data_ptr()


def _workspace(ws, index):
    """A caller's workspace: the library sees its address and size alone."""
    if ws.get_device() != index or not ws.is_contiguous():
        raise ValueError(f"ws: needs packed memory on cuda:{index}")


class _NormShape:
    """What a layer norm call needs to know of the shapes and strides of its fields: worked out
    once for each combination, as a plan's is."""

    def __init__(self, dtype, shape, x_stride, y_stride, gx_stride, eps):
        if len(shape) < 2:
            raise ValueError("layer norm: x is [batch, channels, *grid]")
        if dtype not in _KINDS:
            raise ValueError(f"float32, bfloat16 or float16 data expected, not {dtype}")
        npts = 1
        for n in shape[2:]:
            npts *= n
        batch = [self._batch_stride(shape, st, name) for st, name in
                 ((x_stride, "x"), (y_stride, "y or grad_y"), (gx_stride, "grad_x"))]
        self.desc = fno_layer_norm_desc(_KINDS[dtype], 0, shape[0], shape[1], npts, *batch, eps)
        self.ptr = byref(self.desc)
        self.channels = shape[1:2]
        self.stats = (2, shape[0]) + shape[2:]
        self.ws_bytes = fno_layer_norm_workspace_bytes(self.desc)

    @staticmethod
    def _batch_stride(shape, stride, name):
        """Elements between the batch entries of a field whose entries have to be packed."""
        packed = 1
        if 0 not in shape:
            for n, st in zip(shape[:0:-1], stride[:0:-1]):
                if n != 1 and st != packed:
                    raise ValueError(f"{name}: its batch entries must be packed "
                                     "(call .contiguous())")
                packed *= n
        return stride[0] if shape[0] > 1 else packed


_norm_shape = functools.lru_cache(maxsize=256)(_NormShape)


def _on_gpu(x):
    index = x.get_device()
    if index < 0:
        raise ValueError(f"tensors on the GPU expected, not on {x.device}")
    return index


def _like_x(t, x, name):
    if t.shape != x.shape or t.dtype != x.dtype or t.get_device() != x.get_device():
        raise ValueError(f"{name}: needs x's shape, dtype and device, {tuple(x.shape)} "
                         f"{x.dtype} on {x.device}")
    return t.stride()


def layer_norm_fwd(x, gamma=None, beta=None, eps=1e-5, out=None, stats=None, want_stats=True):
    """Layer norm of a field [B, C, *grid] over its channels at each point ([rows, C]: over each
    row), times gamma plus beta (float32 [C]; None: 1 and 0).  Returns (y, stats); stats, float32
    [2, B, *grid], holds the means and the reciprocal deviations for layer_norm_bwd (None without
    want_stats)."""
    strides = x.stride()
    if out is None:
        out = x.new_empty(x.shape)
        y_strides = out.stride()
    else:
        y_strides = _like_x(out, x, "out")
    n = _norm_shape(x.dtype, x.shape, strides, y_strides, y_strides, eps)
    index = _on_gpu(x)
    if stats is None and want_stats:
        stats = x.new_empty(n.stats, dtype=_torch.float32)
    _check(_on_stream(index, _lib.fno_layer_norm_fwd, n.ptr, x.data_ptr(),
                      _vector(gamma, n.channels, index, "gamma"),
                      _vector(beta, n.channels, index, "beta"), out.data_ptr(),
                      _vector(stats, n.stats, index, "stats")), "fno_layer_norm_fwd")
    return out, stats


def layer_norm_bwd(x, gamma, stats, grad_y, want=("x", "gamma", "beta"), out=None, ws=None):
    """Gradients of layer_norm_fwd from its x and stats: dict(x, gamma, beta), None where not
    asked.  out: tensors to write instead of new ones (out["x"] may be grad_y itself).  ws: packed
    workspace of fno_layer_norm_workspace_bytes on x's device (allocated when None)."""
    gy_strides = _like_x(grad_y, x, "grad_y")
    o = out or {}
    gx = o["x"] if "x" in o else x.new_empty(x.shape) if "x" in want else None
    n = _norm_shape(x.dtype, x.shape, x.stride(), gy_strides,
                    gy_strides if gx is None else _like_x(gx, x, "grad_x"), 0.0)
    index = _on_gpu(x)
    gg, gb = (o[k] if k in o else x.new_empty(n.channels, dtype=_torch.float32) if k in want
              else None for k in ("gamma", "beta"))
    if ws is None:
        ws = x.new_empty(n.ws_bytes, dtype=_torch.uint8) if n.ws_bytes else None
    else:
        _workspace(ws, index)
    _check(_on_stream(index, _lib.fno_layer_norm_bwd, n.ptr, x.data_ptr(),
                      _vector(gamma, n.channels, index, "gamma"),
                      _vector(stats, n.stats, index, "stats"), grad_y.data_ptr(), _ptr(gx),
                      _vector(gg, n.channels, index, "grad_gamma"),
                      _vector(gb, n.channels, index, "grad_beta"), _ptr(ws),
                      0 if ws is None else ws.numel() * ws.element_size()), "fno_layer_norm_bwd")
    return {"x": gx, "gamma": gg, "beta": gb}


class TensorList:
    """Tensors that one call goes over (gradients, parameters, moments): packed float32,
    bfloat16, float16 or complex64 tensors on one GPU.  Made once for buffers that stay: it holds
    the tensors, and uploads the table of their addresses on the current stream.  Functions that
    take a TensorList also take a plain sequence, and make a list for the one call (13 us for 5
    tensors, 209 for 301).  A tensor that a call writes is listed once."""

    def __init__(self, tensors):
        self.handle = None
        self.tensors = list(tensors)
        self.device = self.tensors[0].device if self.tensors else \
            _torch.device("cuda", _torch.cuda.current_device())
        self.index = _torch.cuda.current_device() if self.device.index is None and \
            self.device.type == "cuda" else self.device.index
        entries = (fno_tensor * max(len(self.tensors), 1))()
        for i, t in enumerate(self.tensors):
            if not t.is_contiguous() or t.is_conj() or t.is_neg():
                raise ValueError(f"tensor {i} of the list is not packed (call .contiguous())")
            if t.device != self.device or not t.is_cuda:
                raise ValueError("the tensors of a list are on one GPU")
            if t.dtype not in _LIST_KINDS:
                raise ValueError(f"float32, bfloat16 or float16 data expected, not {t.dtype}")
            e = entries[i]
            e.data, e.dtype = t.data_ptr(), _LIST_KINDS[t.dtype]
            e.elems = 2 * t.numel() if t.is_complex() else t.numel()
        count = len(self.tensors)
        ptr = ctypes.addressof(entries)
        self.table = _torch.empty(max(fno_tensor_list_bytes(count, ptr), 16), dtype=_torch.uint8,
                                  device=self.device)

        def create(stream):
            return fno_tensor_list_create(count, ptr, self.table.data_ptr(), self.table.numel(),
                                          stream)

        self.handle = _on_stream(self.index, create)
        self.norm_ws_bytes = fno_grad_norm_workspace_bytes(self.handle)

    def __len__(self):
        return len(self.tensors)

    def close(self):
        if getattr(self, "handle", None):
            fno_tensor_list_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _tensor_list(ts):
    return ts if isinstance(ts, TensorList) else TensorList(ts)


def _norm_buffers(gl, record, ws):
    if record is None:
        record = gl.table.new_empty(2, dtype=_torch.float32)
    else:
        _vector(record, _RECORD, gl.index, "record")
    if ws is None:
        ws = gl.table.new_empty(gl.norm_ws_bytes)
    else:
        _workspace(ws, gl.index)
    return record, ws


_RECORD = _torch.Size([2])


def grad_norm(grads, max_norm=float("inf"), grad_scale=1.0, record=None, ws=None):
    """The global norm of a list of gradients, which carry the loss scale grad_scale, and what
    clipping to max_norm multiplies them by: a device tensor record = [norm, factor] (see
    fno_grad_norm)."""
    gl = _tensor_list(grads)
    record, ws = _norm_buffers(gl, record, ws)
    _check(_on_stream(gl.index, _lib.fno_grad_norm, gl.handle, max_norm, grad_scale,
                      record.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size()),
           "fno_grad_norm")
    return record


def clip_grad_norm(grads, max_norm, grad_scale=1.0, out=None, record=None, ws=None):
    """grad_norm, and every gradient times the factor, in place or into the tensors of `out` (of
    the gradient's dtype or float32).  Returns the record [norm, factor]."""
    gl = _tensor_list(grads)
    ol = gl if out is None else _tensor_list(out)
    record, ws = _norm_buffers(gl, record, ws)
    _check(_on_stream(gl.index, _lib.fno_clip_grad_norm, gl.handle, ol.handle, max_norm,
                      grad_scale, record.data_ptr(), ws.data_ptr(),
                      ws.numel() * ws.element_size()), "fno_clip_grad_norm")
    return record


def adamw(params, grads, exp_avg, exp_avg_sq, step, lr, betas=(0.9, 0.999), eps=1e-8,
          weight_decay=0.01, record=None):
    """One AdamW update, number `step` (from 1), of float32 (or complex64, as pairs) parameters in
    place, from gradients times the factor of `record` (grad_norm's; None: as they are).  A factor
    that is not finite leaves parameters and moments as they are.  A captured call replays this
    step's number and lr."""
    pl, gl, ml, vl = (_tensor_list(params), _tensor_list(grads), _tensor_list(exp_avg),
                      _tensor_list(exp_avg_sq))
    d = fno_adamw_desc(lr, betas[0], betas[1], eps, weight_decay, step)
    _check(_on_stream(pl.index, _lib.fno_adamw, pl.handle, gl.handle, ml.handle, vl.handle,
                      byref(d), _vector(record, _RECORD, pl.index, "record")), "fno_adamw")
