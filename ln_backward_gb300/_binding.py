"""ctypes binding over libtb.so -- argument marshalling only.

Every function here carries the name of the C entry point it calls, turns
torch tensors into (pointer, size, dtype) arguments, passes torch's current
CUDA stream unless one is given, and raises ``TbError`` on a non-OK status.
No arithmetic of the kernels happens in Python, and there is no fallback:
if libtb.so is missing, importing this module fails.
"""
from __future__ import annotations

import ctypes
import os
import struct
from array import array
from typing import Optional, Sequence

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libtb.so")

TB_F32, TB_F16, TB_BF16 = 0, 1, 2
_DTYPE = {torch.float32: TB_F32, torch.float16: TB_F16, torch.bfloat16: TB_BF16}

STATUS = {0: "TB_OK", 1: "TB_ERR_INVALID_VALUE", 2: "TB_ERR_UNSUPPORTED_DTYPE",
          3: "TB_ERR_MISALIGNED", 4: "TB_ERR_ALIAS", 5: "TB_ERR_WORKSPACE", 6: "TB_ERR_OOM",
          7: "TB_ERR_CUDA", 8: "TB_ERR_DEVICE", 9: "TB_ERR_TIMEOUT"}

# Every symbol include/tb.h declares.
EXPORTS = ("tb_status_string", "tb_version", "tb_device_error", "tb_adamw_plan_create",
           "tb_adamw_step", "tb_adamw_plan_destroy", "tb_softmax_bwd",
           "tb_layernorm_bwd_workspace_size", "tb_layernorm_bwd", "tb_layernorm_bwd_noalloc",
           "tb_softmax_bwd_causal", "tb_rmsnorm_bwd_workspace_size", "tb_rmsnorm_bwd",
           "tb_adamw_grad_norm_workspace_size", "tb_adamw_grad_norm", "tb_adamw_step_clipped",
           "tb_cast_to_f32", "tb_cast_from_f32", "tb_layernorm_bwd_selftest_timeout",
           "tb_adamw_step_device", "tb_adamw_selftest_stale_counter", "tb_rope_freqs", "tb_rope",
           "tb_rope_bwd", "tb_qk_norm_rope", "tb_qk_norm_rope_bwd_workspace_size",
           "tb_qk_norm_rope_bwd", "tb_linear_xent_workspace_size", "tb_linear_xent",
           "tb_linear_xent_bwd_workspace_size", "tb_linear_xent_bwd",
           "tb_linear_xent_selftest_timeout", "tb_gated_linear_workspace_size", "tb_gated_linear",
           "tb_gated_linear_bwd_workspace_size", "tb_gated_linear_bwd", "tb_attention",
           "tb_attention_bwd_workspace_size", "tb_attention_bwd", "tb_attention_selftest_timeout",
           "tb_gated_linear_selftest_timeout")


class TbError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {STATUS.get(code, code)}")
        self.code = code


class tb_tensor_desc(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("grad", ctypes.c_void_p), ("copy", ctypes.c_void_p), ("n", ctypes.c_int64)]


class tb_adamw_hparams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float)]


class tb_heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride_batch", ctypes.c_int64),
                ("stride_seq", ctypes.c_int64), ("stride_head", ctypes.c_int64),
                ("heads", ctypes.c_int64)]


class tb_rope_angles(ctypes.Structure):
    _fields_ = [("freqs", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("positions_stride", ctypes.c_int64), ("offset", ctypes.c_int64),
                ("rotary_dim", ctypes.c_int), ("layout", ctypes.c_int),
                ("magnitude", ctypes.c_float)]


class tb_rope_scaling(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("factor", ctypes.c_double),
                ("original_context", ctypes.c_double), ("fast", ctypes.c_double),
                ("slow", ctypes.c_double)]


def _load_library(path: str = _LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise ImportError(f"{path} is not built; run `python -c 'import __graft_entry__ as g; "
                          "g.build()'` (needs nvcc) -- there is no CPU fallback")
    lib = ctypes.CDLL(path)
    vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    lib.tb_status_string.argtypes = [i32]
    lib.tb_status_string.restype = ctypes.c_char_p
    lib.tb_version.argtypes = []
    lib.tb_version.restype = i32
    lib.tb_device_error.argtypes = [ctypes.POINTER(i32), i32]
    lib.tb_device_error.restype = i32
    lib.tb_adamw_plan_create.argtypes = [ctypes.POINTER(tb_tensor_desc), i32, i32, i32,
                                         ctypes.POINTER(vp)]
    lib.tb_adamw_plan_create.restype = i32
    lib.tb_adamw_step.argtypes = [vp, i64, ctypes.POINTER(tb_adamw_hparams), f32, vp]
    lib.tb_adamw_step.restype = i32
    lib.tb_adamw_plan_destroy.argtypes = [vp]
    lib.tb_adamw_plan_destroy.restype = i32
    lib.tb_softmax_bwd.argtypes = [vp, vp, vp, i64, i64, i32, vp]
    lib.tb_softmax_bwd.restype = i32
    lib.tb_layernorm_bwd_workspace_size.argtypes = [i64, i64, i32, ctypes.POINTER(ctypes.c_size_t)]
    lib.tb_layernorm_bwd_workspace_size.restype = i32
    lib.tb_layernorm_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i32, vp,
                                     ctypes.c_size_t, vp]
    lib.tb_layernorm_bwd.restype = i32
    lib.tb_layernorm_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i32, vp]
    lib.tb_layernorm_bwd_noalloc.restype = i32
    lib.tb_softmax_bwd_causal.argtypes = [vp, vp, vp, i64, i64, i64, i64, i32, vp]
    lib.tb_softmax_bwd_causal.restype = i32
    lib.tb_rmsnorm_bwd_workspace_size.argtypes = [i64, i64, i32, ctypes.POINTER(ctypes.c_size_t)]
    lib.tb_rmsnorm_bwd_workspace_size.restype = i32
    lib.tb_rmsnorm_bwd.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i32, vp, ctypes.c_size_t, vp]
    lib.tb_rmsnorm_bwd.restype = i32
    lib.tb_adamw_grad_norm_workspace_size.argtypes = [vp, ctypes.POINTER(ctypes.c_size_t)]
    lib.tb_adamw_grad_norm_workspace_size.restype = i32
    lib.tb_adamw_grad_norm.argtypes = [vp, f32, f32, vp, vp, ctypes.c_size_t, vp]
    lib.tb_adamw_grad_norm.restype = i32
    lib.tb_adamw_step_clipped.argtypes = [vp, i64, ctypes.POINTER(tb_adamw_hparams), f32, vp, vp]
    lib.tb_adamw_step_clipped.restype = i32
    lib.tb_cast_to_f32.argtypes = [vp, i32, f32, vp, i64, vp]
    lib.tb_cast_to_f32.restype = i32
    lib.tb_cast_from_f32.argtypes = [vp, vp, i32, i64, vp]
    lib.tb_cast_from_f32.restype = i32
    lib.tb_adamw_step_device.argtypes = [vp, vp, ctypes.POINTER(tb_adamw_hparams), f32, vp, vp]
    lib.tb_adamw_step_device.restype = i32
    lib.tb_layernorm_bwd_selftest_timeout.argtypes = [i64, vp]
    lib.tb_layernorm_bwd_selftest_timeout.restype = i32
    lib.tb_linear_xent_selftest_timeout.argtypes = [i64, ctypes.POINTER(i32), vp]
    lib.tb_linear_xent_selftest_timeout.restype = i32
    for fn in (lib.tb_attention_selftest_timeout, lib.tb_gated_linear_selftest_timeout):
        fn.argtypes = [i64, ctypes.POINTER(i32), vp]
        fn.restype = i32
    lib.tb_adamw_selftest_stale_counter.argtypes = [vp, ctypes.c_uint64, vp]
    lib.tb_adamw_selftest_stale_counter.restype = i32
    # tb_heads* and tb_rope_angles*: the binding passes addresses into one packed array
    heads = angles = vp
    lib.tb_rope_freqs.argtypes = [i32, ctypes.c_double, ctypes.POINTER(tb_rope_scaling), vp,
                                  ctypes.POINTER(f32)]
    lib.tb_rope_freqs.restype = i32
    for fn in (lib.tb_rope, lib.tb_rope_bwd):
        fn.argtypes = [heads, heads, heads, heads, i64, i64, i64, angles, i32, vp]
        fn.restype = i32
    lib.tb_qk_norm_rope.argtypes = [heads, heads, vp, vp, f32, heads, heads, vp, vp, i64, i64, i64,
                                    angles, i32, vp]
    lib.tb_qk_norm_rope.restype = i32
    lib.tb_qk_norm_rope_bwd_workspace_size.argtypes = [i64, i64, i64, i64, i64, i32,
                                                       ctypes.POINTER(ctypes.c_size_t)]
    lib.tb_qk_norm_rope_bwd_workspace_size.restype = i32
    lib.tb_qk_norm_rope_bwd.argtypes = [heads, heads, heads, heads, vp, vp, vp, vp, heads, heads,
                                        vp, vp, i64, i64, i64, angles, i32, vp, ctypes.c_size_t, vp]
    lib.tb_qk_norm_rope_bwd.restype = i32
    for fn in (lib.tb_linear_xent_workspace_size, lib.tb_linear_xent_bwd_workspace_size):
        fn.argtypes = [i64, i64, i64, i32, ctypes.POINTER(ctypes.c_size_t)]
        fn.restype = i32
    lib.tb_linear_xent.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, i32, vp, ctypes.c_size_t, vp]
    lib.tb_linear_xent.restype = i32
    lib.tb_linear_xent_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i32, vp,
                                       ctypes.c_size_t, vp]
    lib.tb_linear_xent_bwd.restype = i32
    lib.tb_attention.argtypes = [heads, heads, heads, heads, vp, i64, i64, i64, vp, i64, f32, i32, vp]
    lib.tb_attention.restype = i32
    lib.tb_attention_bwd_workspace_size.argtypes = [i64, i64, i64, i64, i64, i32,
                                                    ctypes.POINTER(ctypes.c_size_t)]
    lib.tb_attention_bwd_workspace_size.restype = i32
    lib.tb_attention_bwd.argtypes = ([heads] * 5 + [vp] + [heads] * 3 +
                                     [i64, i64, i64, vp, i64, f32, i32, vp, ctypes.c_size_t, vp])
    lib.tb_attention_bwd.restype = i32
    for fn in (lib.tb_gated_linear_workspace_size, lib.tb_gated_linear_bwd_workspace_size):
        fn.argtypes = [i64, i64, i64, i32, ctypes.POINTER(ctypes.c_size_t)]
        fn.restype = i32
    lib.tb_gated_linear.argtypes = [vp] * 6 + [i64, i64, i64, i32, i32, vp, ctypes.c_size_t, vp]
    lib.tb_gated_linear.restype = i32
    lib.tb_gated_linear_bwd.argtypes = [vp] * 9 + [i64, i64, i64, i32, i32, vp, ctypes.c_size_t, vp]
    lib.tb_gated_linear_bwd.restype = i32
    return lib


lib = _load_library()


def library_path() -> str:
    return _LIB_PATH


def _check(fn: str, code: int) -> None:
    if code != 0:
        raise TbError(fn, code)


# What torch.cuda.current_device() and current_stream() call, without the lazy initialisation
# (a CUDA tensor exists by then) and the Stream object: a microsecond or two less per call.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> Optional[int]:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    """Device pointer of a contiguous CUDA tensor on the current device (the C entry
    points take device pointers and launch on the current device)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors passed to libtb must be CUDA tensors")
    if t.get_device() != _current_device():
        raise ValueError(f"tensor on {t.device}, but the current device is "
                         f"cuda:{_current_device()}")
    if not t.is_contiguous():
        raise ValueError("tensors passed to libtb must be contiguous")
    return t.data_ptr() if t.numel() > 0 else (t.data_ptr() or None)


def _want(t: torch.Tensor, n: int, dtype: torch.dtype, name: str) -> None:
    """The kernels index `t` by the sizes of the other arguments: check it holds them."""
    if t.numel() != n or t.dtype != dtype:
        raise ValueError(f"{name} must hold {n} {dtype} values, got {t.numel()} {t.dtype}")


def _dtype(t: torch.Tensor) -> int:
    try:
        return _DTYPE[t.dtype]
    except KeyError:
        raise TbError("dtype", 2) from None


# ----------------------------------------------------------------------------- misc
def tb_status_string(code: int) -> str:
    return lib.tb_status_string(int(code)).decode()


def tb_version() -> int:
    return lib.tb_version()


def tb_device_error(reset: bool = True) -> int:
    """Device-side error word of the current device (0: no kernel gave up)."""
    code = ctypes.c_int(0)
    _check("tb_device_error", lib.tb_device_error(ctypes.byref(code), int(reset)))
    return code.value


def tb_layernorm_bwd_selftest_timeout(wait_limit_ns: int = 2_000_000, stream=None) -> None:
    """Runs the LayerNorm ring kernel with its copies withheld so that its bounded
    waits run out; synchronises. tb_device_error() then reports TB_ERR_TIMEOUT."""
    _check("tb_layernorm_bwd_selftest_timeout",
           lib.tb_layernorm_bwd_selftest_timeout(int(wait_limit_ns), _stream(stream)))


TB_LINEAR_XENT_SELFTEST_LAUNCHES = 11


def tb_linear_xent_selftest_timeout(wait_limit_ns: int = 2_000_000, stream=None) -> int:
    """Runs the output layer's product on one pair of CTAs, TB_LINEAR_XENT_SELFTEST_LAUNCHES times with
    something withheld, so that its bounded waits run out; synchronises. Returns the number of launches
    that gave up; tb_device_error() then reports TB_ERR_TIMEOUT."""
    launches = ctypes.c_int(0)
    _check("tb_linear_xent_selftest_timeout",
           lib.tb_linear_xent_selftest_timeout(int(wait_limit_ns), ctypes.byref(launches), _stream(stream)))
    return launches.value


TB_ATTENTION_SELFTEST_LAUNCHES, TB_GATED_LINEAR_SELFTEST_LAUNCHES = 30, 8


def tb_attention_selftest_timeout(wait_limit_ns: int = 2_000_000, stream=None) -> int:
    """The same for attention's kernels: TB_ATTENTION_SELFTEST_LAUNCHES launches."""
    launches = ctypes.c_int(0)
    _check("tb_attention_selftest_timeout",
           lib.tb_attention_selftest_timeout(int(wait_limit_ns), ctypes.byref(launches), _stream(stream)))
    return launches.value


def tb_gated_linear_selftest_timeout(wait_limit_ns: int = 2_000_000, stream=None) -> int:
    """The same for the gated projections' products: TB_GATED_LINEAR_SELFTEST_LAUNCHES launches."""
    launches = ctypes.c_int(0)
    _check("tb_gated_linear_selftest_timeout",
           lib.tb_gated_linear_selftest_timeout(int(wait_limit_ns), ctypes.byref(launches), _stream(stream)))
    return launches.value


# ----------------------------------------------------------------------------- AdamW
class AdamWPlan:
    """Owns a ``tb_adamw_plan*``; keeps the tensors it points at alive."""

    def __init__(self, handle: int, tensors):
        self.handle = handle
        self._keep = tensors

    def close(self) -> None:
        if self.handle:
            _check("tb_adamw_plan_destroy", lib.tb_adamw_plan_destroy(self.handle))
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def tb_adamw_plan_create(params: Sequence[torch.Tensor], ms: Sequence[torch.Tensor],
                         vs: Sequence[torch.Tensor], grads: Sequence[torch.Tensor],
                         copies: Sequence[torch.Tensor]) -> AdamWPlan:
    n = len(params)
    if not (len(ms) == len(vs) == len(grads) == len(copies) == n):
        raise ValueError("params, m, v, grads and copies must have one entry per tensor")
    gdtype = grads[0].dtype if n else None
    cdtypes = {c.dtype for c in copies if c is not None}
    if len(cdtypes) > 1:
        raise ValueError("every working copy must have the same dtype")
    for i in range(n):
        k = params[i].numel()
        _want(params[i], k, torch.float32, f"params[{i}]")
        _want(ms[i], k, torch.float32, f"m[{i}]")
        _want(vs[i], k, torch.float32, f"v[{i}]")
        _want(grads[i], k, gdtype, f"grads[{i}]")
        if copies[i] is not None:
            _want(copies[i], k, copies[i].dtype, f"copies[{i}]")
    descs = (tb_tensor_desc * max(n, 1))()
    for i in range(n):
        descs[i] = tb_tensor_desc(_ptr(params[i]), _ptr(ms[i]), _ptr(vs[i]), _ptr(grads[i]),
                                  _ptr(copies[i]), params[i].numel())
    gdt = _dtype(grads[0]) if n else TB_BF16
    with_copy = [c for c in copies if c is not None]
    cdt = _dtype(with_copy[0]) if with_copy else TB_BF16
    handle = ctypes.c_void_p(None)
    _check("tb_adamw_plan_create",
           lib.tb_adamw_plan_create(descs, n, gdt, cdt, ctypes.byref(handle)))
    return AdamWPlan(handle.value, (list(params), list(ms), list(vs), list(grads), list(copies)))


def tb_adamw_step(plan: AdamWPlan, step: int, lr: float, beta1: float, beta2: float, eps: float,
                  weight_decay: float, inv_loss_scale: float, stream=None) -> None:
    hp = tb_adamw_hparams(lr, beta1, beta2, eps, weight_decay)
    _check("tb_adamw_step", lib.tb_adamw_step(plan.handle, int(step), ctypes.byref(hp),
                                              float(inv_loss_scale), _stream(stream)))


def tb_adamw_step_device(plan: AdamWPlan, step: torch.Tensor, lr: float, beta1: float, beta2: float,
                         eps: float, weight_decay: float, inv_loss_scale: float,
                         clip: Optional[torch.Tensor] = None, stream=None) -> None:
    """The step counter is a 1-element int64 CUDA tensor, read when the kernel runs."""
    if step.dtype != torch.int64 or step.numel() != 1 or not step.is_cuda:
        raise ValueError("step must be a 1-element int64 CUDA tensor")
    if clip is not None and (clip.dtype != torch.float32 or clip.numel() < 3):
        raise ValueError("clip must hold 3 fp32 values")
    hp = tb_adamw_hparams(lr, beta1, beta2, eps, weight_decay)
    _check("tb_adamw_step_device",
           lib.tb_adamw_step_device(plan.handle, _ptr(step), ctypes.byref(hp), float(inv_loss_scale),
                                    _ptr(clip), _stream(stream)))


def tb_adamw_plan_destroy(plan: AdamWPlan) -> None:
    plan.close()


def tb_adamw_selftest_stale_counter(plan: AdamWPlan, next_tile: int, stream=None) -> None:
    """Test hook: leaves a stale value in the plan's tile counter (synchronises)."""
    _check("tb_adamw_selftest_stale_counter",
           lib.tb_adamw_selftest_stale_counter(plan.handle, int(next_tile), _stream(stream)))


def tb_adamw_grad_norm_workspace_size(plan: AdamWPlan) -> int:
    out = ctypes.c_size_t(0)
    _check("tb_adamw_grad_norm_workspace_size",
           lib.tb_adamw_grad_norm_workspace_size(plan.handle, ctypes.byref(out)))
    return out.value


def tb_adamw_grad_norm(plan: AdamWPlan, inv_loss_scale: float, max_norm: float,
                       out: torch.Tensor, workspace: torch.Tensor, stream=None) -> None:
    """Writes {norm, clip factor, nonfinite} (3 fp32 values) into ``out`` on the device."""
    if out.dtype != torch.float32 or out.numel() < 3:
        raise ValueError("out must hold 3 fp32 values")
    _check("tb_adamw_grad_norm",
           lib.tb_adamw_grad_norm(plan.handle, float(inv_loss_scale), float(max_norm), _ptr(out),
                                  _ptr(workspace), workspace.numel() * workspace.element_size(),
                                  _stream(stream)))


def tb_adamw_step_clipped(plan: AdamWPlan, step: int, lr: float, beta1: float, beta2: float,
                          eps: float, weight_decay: float, inv_loss_scale: float,
                          clip: torch.Tensor, stream=None) -> None:
    """tb_adamw_step with the gradient scaled by clip[1]; skipped when clip[2] != 0."""
    if clip.dtype != torch.float32 or clip.numel() < 3:
        raise ValueError("clip must hold 3 fp32 values")
    hp = tb_adamw_hparams(lr, beta1, beta2, eps, weight_decay)
    _check("tb_adamw_step_clipped",
           lib.tb_adamw_step_clipped(plan.handle, int(step), ctypes.byref(hp), float(inv_loss_scale),
                                     _ptr(clip), _stream(stream)))


# ----------------------------------------------------------------------------- casts
def tb_cast_to_f32(src: torch.Tensor, dst: torch.Tensor, scale: float = 1.0, stream=None) -> None:
    """dst = float(src) * scale (dst fp32, same number of elements)."""
    if dst.dtype != torch.float32 or dst.numel() != src.numel():
        raise ValueError("dst must be fp32 with as many elements as src")
    _check("tb_cast_to_f32", lib.tb_cast_to_f32(_ptr(src), _dtype(src), float(scale), _ptr(dst),
                                                src.numel(), _stream(stream)))


def tb_cast_from_f32(src: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
    """dst = round-to-nearest-even(src) in dst's 16-bit dtype."""
    if src.dtype != torch.float32 or dst.numel() != src.numel():
        raise ValueError("src must be fp32 with as many elements as dst")
    _check("tb_cast_from_f32", lib.tb_cast_from_f32(_ptr(src), _ptr(dst), _dtype(dst), src.numel(),
                                                    _stream(stream)))


# ----------------------------------------------------------------------------- softmax bwd
def tb_softmax_bwd(dY: torch.Tensor, P: torch.Tensor, dX: torch.Tensor, stream=None) -> None:
    """dX = P * (dY - rowsum(P*dY)) over the last dimension of [rows, cols] tensors."""
    if not (dY.shape == P.shape == dX.shape) or dY.dim() != 2:
        raise ValueError("dY, P and dX must be [rows, cols] tensors of one shape")
    if not (dY.dtype == P.dtype == dX.dtype):
        raise ValueError("dY, P and dX must share a dtype")
    rows, cols = dY.shape
    _check("tb_softmax_bwd", lib.tb_softmax_bwd(_ptr(dY), _ptr(P), _ptr(dX), rows, cols,
                                                _dtype(dY), _stream(stream)))


def tb_softmax_bwd_causal(dY: torch.Tensor, P: torch.Tensor, dX: torch.Tensor, period: int,
                          offset: int = 0, stream=None) -> None:
    """Softmax backward reading only the causally open columns of each row:
    row r is nonzero only on its first min(cols, r % period + 1 + offset) columns."""
    if not (dY.shape == P.shape == dX.shape) or dY.dim() != 2:
        raise ValueError("dY, P and dX must be [rows, cols] tensors of one shape")
    if not (dY.dtype == P.dtype == dX.dtype):
        raise ValueError("dY, P and dX must share a dtype")
    rows, cols = dY.shape
    _check("tb_softmax_bwd_causal",
           lib.tb_softmax_bwd_causal(_ptr(dY), _ptr(P), _ptr(dX), rows, cols, int(period),
                                     int(offset), _dtype(dY), _stream(stream)))


# ----------------------------------------------------------------------------- RMSNorm bwd
def tb_rmsnorm_bwd_workspace_size(rows: int, D: int, dtype: torch.dtype) -> int:
    out = ctypes.c_size_t(0)
    _check("tb_rmsnorm_bwd_workspace_size",
           lib.tb_rmsnorm_bwd_workspace_size(int(rows), int(D), _DTYPE[dtype], ctypes.byref(out)))
    return out.value


def tb_rmsnorm_bwd(dY: torch.Tensor, x: torch.Tensor, inv_rms: torch.Tensor, gamma: torch.Tensor,
                   dX: torch.Tensor, dgamma: torch.Tensor, workspace: Optional[torch.Tensor],
                   stream=None) -> None:
    if x.dim() != 2 or dY.shape != x.shape or dX.shape != x.shape:
        raise ValueError("x, dY and dX must be [rows, D] tensors of one shape")
    if not (dY.dtype == x.dtype == dX.dtype):
        raise ValueError("x, dY and dX must share a dtype")
    rows, D = x.shape
    _want(inv_rms, rows, torch.float32, "inv_rms")
    _want(gamma, D, torch.float32, "gamma")
    _want(dgamma, D, torch.float32, "dgamma")
    ws_ptr = _ptr(workspace) if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("tb_rmsnorm_bwd",
           lib.tb_rmsnorm_bwd(_ptr(dY), _ptr(x), _ptr(inv_rms), _ptr(gamma), _ptr(dX),
                              _ptr(dgamma), rows, D, _dtype(x), ws_ptr, ws_bytes, _stream(stream)))


# ----------------------------------------------------------------------------- LayerNorm bwd
def tb_layernorm_bwd_workspace_size(rows: int, D: int, dtype: torch.dtype) -> int:
    out = ctypes.c_size_t(0)
    _check("tb_layernorm_bwd_workspace_size",
           lib.tb_layernorm_bwd_workspace_size(int(rows), int(D), _DTYPE[dtype], ctypes.byref(out)))
    return out.value


def tb_layernorm_bwd(dY: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, inv_std: torch.Tensor,
                     gamma: torch.Tensor, dX: torch.Tensor, dgamma: torch.Tensor,
                     dbeta: torch.Tensor, workspace: Optional[torch.Tensor], stream=None) -> None:
    if x.dim() != 2 or dY.shape != x.shape or dX.shape != x.shape:
        raise ValueError("x, dY and dX must be [rows, D] tensors of one shape")
    if not (dY.dtype == x.dtype == dX.dtype):
        raise ValueError("x, dY and dX must share a dtype")
    rows, D = x.shape
    _want(mean, rows, torch.float32, "mean")
    _want(inv_std, rows, torch.float32, "inv_std")
    _want(gamma, D, torch.float32, "gamma")
    _want(dgamma, D, torch.float32, "dgamma")
    _want(dbeta, D, torch.float32, "dbeta")
    ws_ptr = _ptr(workspace) if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("tb_layernorm_bwd",
           lib.tb_layernorm_bwd(_ptr(dY), _ptr(x), _ptr(mean), _ptr(inv_std), _ptr(gamma),
                                _ptr(dX), _ptr(dgamma), _ptr(dbeta), rows, D, _dtype(x), ws_ptr,
                                ws_bytes, _stream(stream)))


def tb_layernorm_bwd_noalloc(dY: torch.Tensor, x: torch.Tensor, mean: torch.Tensor,
                             inv_std: torch.Tensor, gamma: torch.Tensor, dX: torch.Tensor,
                             dgamma: torch.Tensor, dbeta: torch.Tensor, stream=None) -> None:
    """tb_layernorm_bwd without a workspace: the library's own fixed scratch array is
    used, nothing is allocated (see include/tb.h for the limits)."""
    if x.dim() != 2 or dY.shape != x.shape or dX.shape != x.shape:
        raise ValueError("x, dY and dX must be [rows, D] tensors of one shape")
    if not (dY.dtype == x.dtype == dX.dtype):
        raise ValueError("x, dY and dX must share a dtype")
    rows, D = x.shape
    _want(mean, rows, torch.float32, "mean")
    _want(inv_std, rows, torch.float32, "inv_std")
    _want(gamma, D, torch.float32, "gamma")
    _want(dgamma, D, torch.float32, "dgamma")
    _want(dbeta, D, torch.float32, "dbeta")
    _check("tb_layernorm_bwd_noalloc",
           lib.tb_layernorm_bwd_noalloc(_ptr(dY), _ptr(x), _ptr(mean), _ptr(inv_std), _ptr(gamma),
                                        _ptr(dX), _ptr(dgamma), _ptr(dbeta), rows, D, _dtype(x),
                                        _stream(stream)))


# ----------------------------------------------------------------------------- rotary positions
ROPE_SCALING = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "wavelength": 4}


def tb_rope_freqs(rotary_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                  original_context: float = 0.0, fast: float = 32.0, slow: float = 1.0,
                  device=None):
    """(freqs, magnitude): an int64 tensor of rotary_dim / 2 frequencies in 2^-64 turn a
    position, on ``device`` (the current CUDA device by default), and the factor on sines and
    cosines. ``scaling``: none, linear, ntk, yarn or wavelength (see include/tb.h)."""
    if scaling not in ROPE_SCALING:
        raise ValueError(f"scaling must be one of {', '.join(ROPE_SCALING)}")
    table = torch.empty(max(int(rotary_dim), 0) // 2, dtype=torch.int64)
    magnitude = ctypes.c_float(0.0)
    how = tb_rope_scaling(ROPE_SCALING[scaling], float(factor), float(original_context),
                          float(fast), float(slow))
    _check("tb_rope_freqs",
           lib.tb_rope_freqs(int(rotary_dim), float(base), ctypes.byref(how),
                             table.data_ptr() or None, ctypes.byref(magnitude)))
    return table.to("cuda" if device is None else device), magnitude.value


_F32 = torch.float32
_HEADS_BYTES = ctypes.sizeof(tb_heads)        # five 8-byte fields
assert _HEADS_BYTES == 40 and ctypes.sizeof(tb_rope_angles) == 48


class _HeadsCall:
    """The tb_heads of a call's tensors and its tb_rope_angles, packed into one array of 64-bit
    words. Small calls take a few microseconds on the GPU, so this path makes no ctypes objects
    and few calls: a struct for each tensor would cost more than the kernel.

    ``tensors`` are the queries, the keys (or None), and pairs behind them with as many heads as
    the queries and the keys."""

    __slots__ = ("words", "p", "batch", "seq", "dim", "code", "device", "heads")

    def __init__(self, names, tensors, freqs: Optional[torch.Tensor],
                 positions: Optional[torch.Tensor], offset: int, interleaved: bool,
                 magnitude: float):
        q = tensors[0]
        shape = q.shape
        if len(shape) != 4:
            raise ValueError(f"{names[0]} must be [batch, seq, heads, head_dim], got {tuple(shape)}")
        batch, seq, _, dim = shape
        dtype, device = q.dtype, q.get_device()
        words, heads = [], []
        for i, t in enumerate(tensors):
            if t is None:
                if i > 1 and heads[i & 1] is not None:
                    raise ValueError(f"{names[i & 1]} and {names[i]} must be given together")
                words += (0, 0, 0, 0, 0)
                heads.append(None)
                continue
            shape = t.shape
            b, s, h, d = shape if len(shape) == 4 else (-1, -1, -1, -1)
            if b != batch or s != seq or d != dim:
                raise ValueError(f"{names[i]} must be [batch, seq, heads, head_dim] with the batch, "
                                 f"seq and head_dim of {names[0]}, got {tuple(shape)}")
            if t.dtype != dtype:
                raise ValueError(f"{names[i]} must be {dtype} like {names[0]}, got {t.dtype}")
            sb, ss, sh, sd = t.stride()
            if sd != 1 and dim > 1:
                raise ValueError(f"the last dimension of {names[i]} must be contiguous")
            if i > 1 and heads[i & 1] != h:
                if heads[i & 1] is None:
                    raise ValueError(f"{names[i & 1]} and {names[i]} must be given together")
                raise ValueError(f"{names[i]} must have {heads[i & 1]} heads, got {h}")
            if t.get_device() != device:
                raise ValueError(f"{names[i]} is on {t.device}, {names[0]} on {q.device}")
            words += (t.data_ptr(), sb, ss, sh, h)
            heads.append(h)
        if device < 0:
            raise ValueError("tensors passed to libtb must be CUDA tensors")
        if device != _current_device():
            raise ValueError(f"tensor on cuda:{device}, but the current device is "
                             f"cuda:{_current_device()}")
        rot = table = where = stride = 0
        if freqs is not None:
            if freqs.dtype != torch.int64 or freqs.dim() != 1 or not freqs.is_contiguous():
                raise ValueError("freqs must be the int64 table of tb_rope_freqs")
            if freqs.get_device() != device:
                raise ValueError(f"freqs is on {freqs.device}, {names[0]} on cuda:{device}")
            rot, table = 2 * freqs.numel(), freqs.data_ptr()
        if positions is not None:
            if positions.dtype != torch.int64 or positions.get_device() != device:
                raise ValueError(f"positions must be an int64 tensor on the device of {names[0]}")
            shape, strides = positions.shape, positions.stride()
            if len(shape) not in (1, 2) or shape[-1] != seq or (len(shape) == 2 and shape[0] != batch):
                raise ValueError(f"positions must be [{batch}, {seq}] or [{seq}], got {tuple(shape)}")
            if seq > 1 and strides[-1] != 1:
                raise ValueError("the last dimension of positions must be contiguous")
            where = positions.data_ptr()
            if len(shape) == 2 and batch > 1:
                stride = strides[0]
        size = _float_bits(magnitude) if magnitude != 1.0 else 0x3F800000
        words += (table, where, stride, int(offset), rot | (bool(interleaved) << 32), size)
        self.words = array("q", words)
        at = self.words.buffer_info()[0]
        # addresses of the tensors' tb_heads (None for one that was not given), the tb_rope_angles last
        self.p = p = [at + i * _HEADS_BYTES for i in range(len(heads) + 1)]
        if None in heads:
            for i, h in enumerate(heads):
                if h is None:
                    p[i] = None
        self.batch, self.seq, self.dim, self.device, self.heads = batch, seq, dim, device, heads
        self.code = _DTYPE.get(dtype)
        if self.code is None:
            raise TbError("dtype", 2)

    def fp32(self, t: Optional[torch.Tensor], n: int, name: str) -> Optional[int]:
        """Address of a contiguous fp32 tensor of n values on the call's device."""
        if t is None:
            raise ValueError(f"{name} is missing")
        if t.numel() != n or t.dtype != _F32:
            _want(t, n, _F32, name)
        if t.get_device() != self.device or not t.is_contiguous():
            return _ptr(t)
        return t.data_ptr() or None

    def stream(self, stream) -> Optional[int]:
        return _raw_stream(self.device) if stream is None and _raw_stream else _stream(stream)


def _float_bits(x: float) -> int:
    return struct.unpack("<i", struct.pack("<f", float(x)))[0] & 0xFFFFFFFF


def tb_rope(q: torch.Tensor, k: Optional[torch.Tensor], q_out: torch.Tensor,
            k_out: Optional[torch.Tensor], freqs: torch.Tensor,
            positions: Optional[torch.Tensor] = None, offset: int = 0, interleaved: bool = False,
            magnitude: float = 1.0, stream=None) -> None:
    """Rotary positions on [batch, seq, heads, head_dim] queries and keys (any strides but the
    last). ``positions``: int64 [batch, seq] or [seq]; None counts from ``offset``. An output
    may be its own input."""
    c = _HeadsCall(("q", "k", "q_out", "k_out"), (q, k, q_out, k_out), freqs, positions, offset,
                   interleaved, magnitude)
    _check("tb_rope", lib.tb_rope(*c.p[:4], c.batch, c.seq, c.dim, c.p[4], c.code, c.stream(stream)))


def tb_rope_bwd(dq_out: torch.Tensor, dk_out: Optional[torch.Tensor], dq: torch.Tensor,
                dk: Optional[torch.Tensor], freqs: torch.Tensor,
                positions: Optional[torch.Tensor] = None, offset: int = 0,
                interleaved: bool = False, magnitude: float = 1.0, stream=None) -> None:
    """Gradient of tb_rope: the transposed rotation of dq_out and dk_out."""
    c = _HeadsCall(("dq_out", "dk_out", "dq", "dk"), (dq_out, dk_out, dq, dk), freqs, positions,
                   offset, interleaved, magnitude)
    _check("tb_rope_bwd", lib.tb_rope_bwd(*c.p[:4], c.batch, c.seq, c.dim, c.p[4], c.code,
                                          c.stream(stream)))


def tb_qk_norm_rope(q: torch.Tensor, k: Optional[torch.Tensor], gamma_q: torch.Tensor,
                    gamma_k: Optional[torch.Tensor], q_out: torch.Tensor,
                    k_out: Optional[torch.Tensor], inv_rms_q: Optional[torch.Tensor] = None,
                    inv_rms_k: Optional[torch.Tensor] = None, eps: float = 1e-6,
                    freqs: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                    offset: int = 0, interleaved: bool = False, magnitude: float = 1.0,
                    stream=None) -> None:
    """RMS norm of every head of q and k, then tb_rope, in one pass. inv_rms_q and inv_rms_k
    (fp32, batch * seq * heads values) receive what tb_qk_norm_rope_bwd needs; leave them out
    when serving. Without ``freqs`` the heads are normalised and not rotated."""
    c = _HeadsCall(("q", "k", "q_out", "k_out"), (q, k, q_out, k_out), freqs, positions, offset,
                   interleaved, magnitude)
    tokens = c.batch * c.seq
    gq = c.fp32(gamma_q, c.dim, "gamma_q")
    gk = None if k is None else c.fp32(gamma_k, c.dim, "gamma_k")
    rq = None if inv_rms_q is None else c.fp32(inv_rms_q, tokens * c.heads[0], "inv_rms_q")
    rk = None if inv_rms_k is None else c.fp32(inv_rms_k, tokens * (c.heads[1] or 0), "inv_rms_k")
    _check("tb_qk_norm_rope",
           lib.tb_qk_norm_rope(c.p[0], c.p[1], gq, gk, float(eps), c.p[2], c.p[3], rq, rk, c.batch,
                               c.seq, c.dim, c.p[4], c.code, c.stream(stream)))


def tb_qk_norm_rope_bwd_workspace_size(batch: int, seq: int, heads_q: int, heads_k: int,
                                       head_dim: int, dtype: torch.dtype) -> int:
    out = ctypes.c_size_t(0)
    _check("tb_qk_norm_rope_bwd_workspace_size",
           lib.tb_qk_norm_rope_bwd_workspace_size(int(batch), int(seq), int(heads_q), int(heads_k),
                                                  int(head_dim), _DTYPE[dtype], ctypes.byref(out)))
    return out.value


def tb_qk_norm_rope_bwd(dq_out: torch.Tensor, dk_out: Optional[torch.Tensor], q: torch.Tensor,
                        k: Optional[torch.Tensor], inv_rms_q: torch.Tensor,
                        inv_rms_k: Optional[torch.Tensor], gamma_q: torch.Tensor,
                        gamma_k: Optional[torch.Tensor], dq: torch.Tensor,
                        dk: Optional[torch.Tensor], dgamma_q: torch.Tensor,
                        dgamma_k: Optional[torch.Tensor], freqs: Optional[torch.Tensor] = None,
                        positions: Optional[torch.Tensor] = None, offset: int = 0,
                        interleaved: bool = False, magnitude: float = 1.0,
                        workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Gradient of tb_qk_norm_rope: dq, dk and the (overwritten) dgamma_q, dgamma_k."""
    c = _HeadsCall(("q", "k", "dq", "dk", "dq_out", "dk_out"), (q, k, dq, dk, dq_out, dk_out), freqs,
                   positions, offset, interleaved, magnitude)
    tokens = c.batch * c.seq
    gq, sq = c.fp32(gamma_q, c.dim, "gamma_q"), c.fp32(dgamma_q, c.dim, "dgamma_q")
    rq = c.fp32(inv_rms_q, tokens * c.heads[0], "inv_rms_q")
    gk = sk = rk = None
    if k is not None:
        gk, sk = c.fp32(gamma_k, c.dim, "gamma_k"), c.fp32(dgamma_k, c.dim, "dgamma_k")
        rk = c.fp32(inv_rms_k, tokens * c.heads[1], "inv_rms_k")
    px, pkx, pdx, pdk, py, pky, angles = c.p
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("tb_qk_norm_rope_bwd",
           lib.tb_qk_norm_rope_bwd(py, pky, px, pkx, rq, rk, gq, gk, pdx, pdk, sq, sk, c.batch, c.seq,
                                   c.dim, angles, c.code, _ptr(workspace), ws_bytes, c.stream(stream)))


# ----------------------------------------------------------------------------- output layer's loss
def _xent_sizes(H: torch.Tensor, W: torch.Tensor, targets: torch.Tensor):
    if H.dim() != 2 or W.dim() != 2 or H.shape[1] != W.shape[1] or H.dtype != W.dtype:
        raise ValueError("H [rows, D] and W [vocab, D] must share D and dtype, got "
                         f"{tuple(H.shape)} {H.dtype} and {tuple(W.shape)} {W.dtype}")
    rows, D = H.shape
    _want(targets, rows, torch.int64, "targets")
    return rows, D, W.shape[0]


def _workspace_size(fn, name: str, *sizes) -> int:
    out = ctypes.c_size_t(0)
    _check(name, fn(*sizes, ctypes.byref(out)))
    return out.value


def tb_linear_xent_workspace_size(rows: int, D: int, vocab: int, dtype: torch.dtype) -> int:
    return _workspace_size(lib.tb_linear_xent_workspace_size, "tb_linear_xent_workspace_size",
                           int(rows), int(D), int(vocab), _DTYPE[dtype])


def tb_linear_xent_bwd_workspace_size(rows: int, D: int, vocab: int, dtype: torch.dtype) -> int:
    return _workspace_size(lib.tb_linear_xent_bwd_workspace_size,
                           "tb_linear_xent_bwd_workspace_size", int(rows), int(D), int(vocab),
                           _DTYPE[dtype])


def tb_linear_xent(H: torch.Tensor, W: torch.Tensor, targets: torch.Tensor, loss: torch.Tensor,
                   lse: torch.Tensor, workspace: Optional[torch.Tensor], ignore_index: int = -100,
                   stream=None) -> None:
    """loss[r] = logsumexp(H[r] W^T) - (H[r] W^T)[targets[r]], without the logits in memory;
    0 where targets[r] is ignore_index. lse receives the log sums for tb_linear_xent_bwd."""
    rows, D, vocab = _xent_sizes(H, W, targets)
    _want(loss, rows, torch.float32, "loss")
    _want(lse, rows, torch.float32, "lse")
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("tb_linear_xent",
           lib.tb_linear_xent(_ptr(H), _ptr(W), _ptr(targets), _ptr(loss), _ptr(lse), rows, D,
                              vocab, int(ignore_index), _dtype(H), _ptr(workspace), ws_bytes,
                              _stream(stream)))


def tb_linear_xent_bwd(dloss: torch.Tensor, H: torch.Tensor, W: torch.Tensor, targets: torch.Tensor,
                       lse: torch.Tensor, dH: Optional[torch.Tensor], dW: Optional[torch.Tensor],
                       workspace: Optional[torch.Tensor], ignore_index: int = -100,
                       stream=None) -> None:
    """Gradients of tb_linear_xent: dH and dW (overwritten; None: not wanted) from dloss, the
    gradient of each row's loss."""
    rows, D, vocab = _xent_sizes(H, W, targets)
    _want(dloss, rows, torch.float32, "dloss")
    _want(lse, rows, torch.float32, "lse")
    if dH is not None:
        _want(dH, rows * D, H.dtype, "dH")
    if dW is not None:
        _want(dW, vocab * D, H.dtype, "dW")
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("tb_linear_xent_bwd",
           lib.tb_linear_xent_bwd(_ptr(dloss), _ptr(H), _ptr(W), _ptr(targets), _ptr(lse), _ptr(dH),
                                  _ptr(dW), rows, D, vocab, int(ignore_index), _dtype(H),
                                  _ptr(workspace), ws_bytes, _stream(stream)))


# ----------------------------------------------------------------------------- attention
_I64 = torch.int64


class _AttentionCall:
    """The tb_heads of a call's tensors, packed as in _HeadsCall: the first has the query heads, and so
    have those numbered in ``like_q``; the others have the key heads. What is right takes one test a tensor
    here; _complain says what is wrong."""

    __slots__ = ("words", "p", "batch", "seq", "dim", "code", "device", "heads_q", "offsets", "sequences",
                 "scale")

    def __init__(self, names, tensors, like_q, offsets: Optional[torch.Tensor], scale: Optional[float]):
        q = tensors[0]
        device, dtype = q.get_device(), q.dtype
        try:
            batch, seq, heads_q, dim = q.shape
            heads_k, words = -1, []
            for i, t in enumerate(tensors):
                b, s, h, d = t.shape
                sb, ss, sh, sd = t.stride()
                if i in like_q:
                    right = h == heads_q
                else:
                    if heads_k < 0:
                        heads_k = h
                    right = h == heads_k
                if not right or b != batch or s != seq or d != dim or sd != 1 and dim > 1 \
                        or t.dtype != dtype or t.get_device() != device:
                    self._complain(names, tensors, like_q)
                words += (t.data_ptr(), sb, ss, sh, h)
        except ValueError:                    # not four dimensions
            self._complain(names, tensors, like_q)
            raise
        if device < 0:
            raise ValueError("tensors passed to libtb must be CUDA tensors")
        if device != _current_device():
            raise ValueError(f"tensor on cuda:{device}, but the current device is "
                             f"cuda:{_current_device()}")
        if offsets is None:
            self.offsets, self.sequences = None, 0
        else:
            self.sequences = offsets.numel() - 1
            if offsets.dtype != _I64 or offsets.dim() != 1 or self.sequences < 0:
                raise ValueError("offsets must hold an int64 for the start of each sequence and one for the last's end")
            if offsets.get_device() != device:
                raise ValueError(f"offsets are on {offsets.device}, {names[0]} on cuda:{device}")
            if not offsets.is_contiguous():
                raise ValueError("tensors passed to libtb must be contiguous")
            self.offsets = offsets.data_ptr()
        self.words = words = array("q", words)
        at = words.buffer_info()[0]
        self.p = range(at, at + len(tensors) * _HEADS_BYTES, _HEADS_BYTES)
        self.batch, self.seq, self.dim, self.device, self.heads_q = batch, seq, dim, device, heads_q
        self.scale = (dim or 1) ** -0.5 if scale is None else scale     # (the library refuses heads of 0)
        self.code = _DTYPE.get(dtype)
        if self.code is None:
            raise TbError("dtype", 2)

    @staticmethod
    def _complain(names, tensors, like_q):
        q = tensors[0]
        if q.dim() != 4:
            raise ValueError(f"{names[0]} must be [batch, seq, heads, head_dim], got {tuple(q.shape)}")
        batch, seq, heads_q, dim = q.shape
        heads_k = None
        for i, t in enumerate(tensors):
            if t.dim() != 4 or t.shape[:2] != q.shape[:2] or t.shape[3] != dim:
                raise ValueError(f"{names[i]} must be [batch, seq, heads, head_dim] with the batch, "
                                 f"seq and head_dim of {names[0]}, got {tuple(t.shape)}")
            if i not in like_q and heads_k is None:
                heads_k = t.shape[2]
            want = heads_q if i in like_q else heads_k
            if t.shape[2] != want:
                raise ValueError(f"{names[i]} must have {want} heads, got {t.shape[2]}")
            if t.dtype != q.dtype:
                raise ValueError(f"{names[i]} must be {q.dtype} like {names[0]}, got {t.dtype}")
            if t.stride(3) != 1 and dim > 1:
                raise ValueError(f"the last dimension of {names[i]} must be contiguous")
            if t.get_device() != q.get_device():
                raise ValueError(f"{names[i]} is on {t.device}, {names[0]} on {q.device}")

    def sums(self, t: torch.Tensor, name: str) -> Optional[int]:
        """Address of a contiguous fp32 [batch, heads_q, seq]."""
        if t.numel() != self.batch * self.heads_q * self.seq or t.dtype != _F32:
            _want(t, self.batch * self.heads_q * self.seq, _F32, name)
        if t.get_device() != self.device or not t.is_contiguous():
            return _ptr(t)
        return t.data_ptr() or None

    def stream(self, stream) -> Optional[int]:
        return _raw_stream(self.device) if stream is None and _raw_stream else _stream(stream)


def tb_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                 lse: Optional[torch.Tensor] = None, offsets: Optional[torch.Tensor] = None,
                 scale: Optional[float] = None, stream=None) -> None:
    """Causal attention of [batch, seq, heads, head_dim] tensors (any strides but the last); k and v
    may have fewer heads than q. ``offsets``: int64, the first token of each of the sequences packed
    into the one row, and the last's end; None: every batch entry is a sequence. lse (fp32
    [batch, heads_q, seq]) receives what tb_attention_bwd needs; leave it out when serving.
    ``scale``: head_dim ** -0.5 by default."""
    c = _AttentionCall(("q", "k", "v", "out"), (q, k, v, out), (0, 3), offsets, scale)
    sums = None if lse is None else c.sums(lse, "lse")
    _check("tb_attention",
           lib.tb_attention(*c.p, sums, c.batch, c.seq, c.dim, c.offsets, c.sequences, c.scale, c.code,
                            c.stream(stream)))


def tb_attention_bwd_workspace_size(batch: int, seq: int, heads_q: int, heads_k: int, head_dim: int,
                                    dtype: torch.dtype) -> int:
    return _workspace_size(lib.tb_attention_bwd_workspace_size, "tb_attention_bwd_workspace_size",
                           int(batch), int(seq), int(heads_q), int(heads_k), int(head_dim),
                           _DTYPE[dtype])


def tb_attention_bwd(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                     out: torch.Tensor, lse: torch.Tensor, dq: torch.Tensor, dk: torch.Tensor,
                     dv: torch.Tensor, workspace: Optional[torch.Tensor],
                     offsets: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                     stream=None) -> None:
    """Gradient of tb_attention: dq, dk and dv (overwritten) from dout, the forward's inputs and
    what it wrote."""
    c = _AttentionCall(("q", "k", "v", "dout", "out", "dq", "dk", "dv"), (q, k, v, dout, out, dq, dk, dv),
                       (0, 3, 4, 5), offsets, scale)
    pq, pk, pv, py, po, gq, gk, gv = c.p
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("tb_attention_bwd",
           lib.tb_attention_bwd(py, pq, pk, pv, po, c.sums(lse, "lse"), gq, gk, gv, c.batch, c.seq, c.dim,
                                c.offsets, c.sequences, c.scale, c.code, _ptr(workspace), ws_bytes,
                                c.stream(stream)))


# ----------------------------------------------------------------------------- gated projections
ACTIVATION = {"silu": 0, "gelu": 1, "gelu_tanh": 2}


def _gated_call(X: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, activation: str, others):
    """(rows, D, F, activation's and dtype's numbers, device, addresses of X, Wg, Wu and of ``others``). Others are
    (tensor or None, its size, its name); sizes are products of rows N, D and F."""
    if X.dim() != 2 or Wg.dim() != 2 or Wg.shape != Wu.shape or X.shape[1] != Wg.shape[1]:
        raise ValueError("X must be [rows, D], Wg and Wu [F, D], got "
                         f"{tuple(X.shape)}, {tuple(Wg.shape)} and {tuple(Wu.shape)}")
    dtype = X.dtype
    if not dtype == Wg.dtype == Wu.dtype:
        raise ValueError("X, Wg and Wu must share a dtype")
    act = ACTIVATION.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATION)}")
    rows, D = X.shape
    F = Wg.shape[0]
    sizes = {"NF": rows * F, "ND": rows * D, "FD": F * D}
    tensors = [X, Wg, Wu]
    for t, size, name in others:
        if t is not None and (t.numel() != sizes[size] or t.dtype != dtype):
            _want(t, sizes[size], dtype, name)
        tensors.append(t)
    device = X.get_device()
    here = device >= 0 and device == _current_device()
    p = [None if t is None else t.data_ptr() or None if here and t.get_device() == device and t.is_contiguous() else _ptr(t)
         for t in tensors]
    return rows, D, F, act, _dtype(X), device, p


def _scratch(workspace: Optional[torch.Tensor]):
    return (None, 0) if workspace is None else (_ptr(workspace), workspace.numel() * workspace.element_size())


def tb_gated_linear_workspace_size(rows: int, D: int, F: int, dtype: torch.dtype) -> int:
    return _workspace_size(lib.tb_gated_linear_workspace_size, "tb_gated_linear_workspace_size",
                           int(rows), int(D), int(F), _DTYPE[dtype])


def tb_gated_linear_bwd_workspace_size(rows: int, D: int, F: int, dtype: torch.dtype) -> int:
    return _workspace_size(lib.tb_gated_linear_bwd_workspace_size,
                           "tb_gated_linear_bwd_workspace_size", int(rows), int(D), int(F),
                           _DTYPE[dtype])


def tb_gated_linear(X: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, H: torch.Tensor,
                    G: Optional[torch.Tensor] = None, U: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, activation: str = "silu",
                    stream=None) -> None:
    """H = act(X Wg^T) * (X Wu^T) in one pass. G and U receive the two products for
    tb_gated_linear_bwd; leave them out when serving."""
    rows, D, F, act, code, device, p = _gated_call(X, Wg, Wu, activation,
                                                   ((H, "NF", "H"), (G, "NF", "G"), (U, "NF", "U")))
    _check("tb_gated_linear",
           lib.tb_gated_linear(*p, rows, D, F, act, code, *_scratch(workspace),
                               _raw_stream(device) if stream is None and _raw_stream else _stream(stream)))


def tb_gated_linear_bwd(dH: torch.Tensor, X: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor,
                        G: torch.Tensor, U: torch.Tensor, dX: Optional[torch.Tensor],
                        dWg: Optional[torch.Tensor], dWu: Optional[torch.Tensor],
                        workspace: Optional[torch.Tensor], activation: str = "silu",
                        stream=None) -> None:
    """Gradients of tb_gated_linear: dX, dWg and dWu (overwritten; None: not wanted) from dH and
    what the forward kept."""
    rows, D, F, act, code, device, p = _gated_call(
        X, Wg, Wu, activation, ((dH, "NF", "dH"), (G, "NF", "G"), (U, "NF", "U"), (dX, "ND", "dX"), (dWg, "FD", "dWg"),
                                (dWu, "FD", "dWu")))
    _check("tb_gated_linear_bwd",
           lib.tb_gated_linear_bwd(p[3], *p[:3], *p[4:], rows, D, F, act, code, *_scratch(workspace),
                                   _raw_stream(device) if stream is None and _raw_stream else _stream(stream)))
