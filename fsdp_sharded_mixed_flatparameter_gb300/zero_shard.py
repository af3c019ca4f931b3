"""ctypes binding of libzeroshard with the C ABI's names.

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  Tensors are PyTorch tensors (device memory and streams come from
PyTorch); they are checked to be contiguous CUDA tensors of the right dtype
before their addresses are handed to the library, so that a host pointer can
never reach a kernel.  There is no CPU fallback: without the built library
every call raises.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import List, NamedTuple, Optional, Sequence, Tuple

import numpy as np
import torch

from . import build as _build

ZERO_OK, ZERO_EINVAL, ZERO_ECUDA = 0, 1, 2
ZERO_F32, ZERO_BF16, ZERO_F16 = 0, 1, 2

_DT = {torch.float32: ZERO_F32, torch.bfloat16: ZERO_BF16, torch.float16: ZERO_F16}


class ZeroError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{msg} (status {status})")
        self.status = status


class zero_tensor(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("numel", ctypes.c_int64), ("flat_offset", ctypes.c_int64)]


class zero_norm_result(ctypes.Structure):
    _fields_ = [("sqnorm", ctypes.c_double), ("norm", ctypes.c_double), ("clip_coef", ctypes.c_float),
                ("finite", ctypes.c_int32)]


class zero_adamw_hparams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double)]


class zero_loss_scale_state(ctypes.Structure):
    _fields_ = [("scale", ctypes.c_float), ("growth_tracker", ctypes.c_int32), ("unscale", ctypes.c_float),
                ("found_inf", ctypes.c_int32)]


class zero_adamw_device_state(ctypes.Structure):
    _fields_ = [("step", ctypes.c_int64), ("apply", ctypes.c_int32), ("status", ctypes.c_int32),
                ("scalars", ctypes.c_float * 8)]


class zero_state8(ctypes.Structure):
    _fields_ = [("exp_avg", ctypes.c_void_p), ("exp_avg_scale", ctypes.c_void_p), ("root", ctypes.c_void_p),
                ("root_scale", ctypes.c_void_p)]


class zero_rounding(ctypes.Structure):
    _fields_ = [("seed", ctypes.c_uint64), ("stream", ctypes.c_int64), ("root_bits", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class zero_list_tensor(ctypes.Structure):
    _fields_ = [("master", ctypes.c_void_p), ("exp_avg", ctypes.c_void_p), ("exp_avg_sq", ctypes.c_void_p),
                ("exp_avg_scale", ctypes.c_void_p), ("root_scale", ctypes.c_void_p), ("lowp", ctypes.c_void_p),
                ("numel", ctypes.c_int64), ("group", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class zero_grad_entry(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("numel", ctypes.c_int64),
                ("src_dtype", ctypes.c_int32), ("dst_dtype", ctypes.c_int32), ("group", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class zero_grad_list(ctypes.Structure):
    _fields_ = [("d_entries", ctypes.c_void_p), ("d_plan", ctypes.c_void_p), ("n_tensors", ctypes.c_int32),
                ("n_groups", ctypes.c_int32), ("n_wide", ctypes.c_int32), ("n_narrow", ctypes.c_int32),
                ("chunk", ctypes.c_int32), ("norm_type", ctypes.c_int32), ("in_place", ctypes.c_int32)]


STATE8_BLOCK = 256      # elements per scale of the 8-bit moments
LIST_CHUNK = 1024       # elements per piece of a tensor list's work
LIST_MAX_GROUPS = 64

NORM_RESULT_BYTES = ctypes.sizeof(zero_norm_result)
HPARAMS_BYTES = ctypes.sizeof(zero_adamw_hparams)
DEVICE_STATE_BYTES = ctypes.sizeof(zero_adamw_device_state)
TENSOR_ENTRY_BYTES = ctypes.sizeof(zero_tensor)
LOSS_SCALE_STATE_BYTES = ctypes.sizeof(zero_loss_scale_state)

_lib = None


def debug_build_selected() -> bool:
    """ZERO_SHARD_DEBUG=1 selects the self-checking debug library (built with -DZERO_DEBUG)."""
    return os.environ.get("ZERO_SHARD_DEBUG", "") == "1"


def library_path() -> str:
    return _build.DEBUG_LIB if debug_build_selected() else _build.LIB


def lib() -> ctypes.CDLL:
    """Load the in-tree libzeroshard.so (built by __graft_entry__.build())."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"libzeroshard is not built ({path} missing): run __graft_entry__.build()")
    L = ctypes.CDLL(path)
    i32, i64, f32, f64, vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_double, ctypes.c_void_p
    L.zero_shard_range.argtypes = [i64, i32, i32, ctypes.POINTER(i64), ctypes.POINTER(i64)]
    L.zero_tensor_table.argtypes = [vp, vp, i32, vp, ctypes.POINTER(i64)]
    sz = ctypes.c_size_t
    L.zero_flatten_cast.argtypes = [vp, i32, i64, ctypes.c_int, i64, i64, f32, vp, i32, vp, vp, vp, sz, vp]
    L.zero_accum.argtypes = [vp, vp, ctypes.c_int, i64, f32, vp, i32, vp, vp, sz, vp]
    L.zero_reduce_chunks.argtypes = [vp, vp, ctypes.c_int, i32, i64, i64, f32, vp, i32, vp, vp, sz, vp]
    L.zero_grad_sqnorm_finalize.argtypes = [vp, i64, f64, f64, vp, vp]
    L.zero_grad_sqnorm_combine.argtypes = [vp, i32, f64, vp, vp]
    L.zero_grad_sqnorm_workspace_bytes.argtypes = [i64]
    L.zero_grad_sqnorm_workspace_bytes.restype = ctypes.c_size_t
    L.zero_grad_sqnorm.argtypes = [vp, i64, f64, f64, vp, ctypes.c_size_t, vp, vp]
    L.zero_grad_sqnorm_noalloc.argtypes = [vp, i64, f64, f64, vp, vp]
    L.zero_adamw_step.argtypes = [vp, vp, vp, vp, vp, ctypes.c_int, i64, ctypes.POINTER(zero_adamw_hparams), i64,
                                  vp, vp]
    L.zero_adamw_step_tensors.argtypes = [vp, vp, vp, vp, i32, i64, ctypes.c_int, i64, f32, vp, vp, vp,
                                          ctypes.c_int, i64, ctypes.POINTER(zero_adamw_hparams), i64, vp, vp]
    L.zero_loss_scale_update.argtypes = [ctypes.POINTER(f32), ctypes.POINTER(i32), i32, f64, f64, i32]
    L.zero_loss_scale_update_device.argtypes = [vp, i32, f64, f64, i32, vp, vp]
    L.zero_adamw_scalars.argtypes = [ctypes.POINTER(zero_adamw_hparams), i64, vp]
    L.zero_debug_errors.argtypes = [vp, i32]
    L.zero_debug_selftest.argtypes = [i64, vp]
    L.zero_adamw_prepare_device.argtypes = [vp, vp, vp, vp]
    L.zero_adamw_step_device.argtypes = [vp, vp, vp, vp, vp, ctypes.c_int, i64, vp, vp, vp]
    L.zero_adamw_step_tensors_device.argtypes = [vp, vp, vp, vp, i32, i64, ctypes.c_int, i64, f32, vp, vp, vp,
                                                 ctypes.c_int, i64, vp, vp, vp]
    hpp, rdp, s8 = ctypes.POINTER(zero_adamw_hparams), ctypes.POINTER(zero_rounding), ctypes.POINTER(zero_state8)
    ci = ctypes.c_int
    L.zero_state8_pack.argtypes = [vp, vp, i64, s8, vp]
    L.zero_state8_unpack.argtypes = [s8, i64, vp, vp, vp]
    L.zero_adamw_step8_tensors.argtypes = [vp, s8, vp, i32, i64, ci, i64, f32, vp, vp, vp, ci, i64, hpp, i64, rdp,
                                           vp, vp]
    L.zero_adamw_step8_tensors_device.argtypes = [vp, s8, vp, i32, i64, ci, i64, f32, vp, vp, vp, ci, i64, vp, rdp,
                                                  vp, vp]
    L.zero_list_chunks.argtypes = [vp, i32, i32, i32, vp, ctypes.POINTER(i32)]
    L.zero_adamw_list.argtypes = [vp, i32, vp, i32, i32, vp, ci, f32, vp, ci, hpp, i32, i64, rdp, vp, vp]
    L.zero_adamw_list_device.argtypes = [vp, i32, vp, i32, i32, vp, ci, f32, vp, ci, vp, i32, rdp, vp, vp]
    L.zero_adamw_list_clips.argtypes = L.zero_adamw_list.argtypes
    L.zero_adamw_list_clips_device.argtypes = L.zero_adamw_list_device.argtypes
    L.zero_adamw_prepare_list_device.argtypes = [vp, i32, vp, vp, vp]
    glp = ctypes.POINTER(zero_grad_list)
    L.zero_grad_plan.argtypes = [vp, vp, i32, i32, vp, glp]
    L.zero_grad_entries_check.argtypes = [vp, vp, i32, i32]
    L.zero_list_norms_workspace_bytes.argtypes = [glp]
    L.zero_list_norms_workspace_bytes.restype = ctypes.c_size_t
    L.zero_list_sums.argtypes = [glp, f32, vp, vp, sz, vp, vp]
    L.zero_sums_norms.argtypes = [glp, vp, i32, vp, vp, vp, vp, vp, vp]
    L.zero_list_clip.argtypes = [glp, f32, vp, vp, vp]
    L.zero_list_norms.argtypes = [glp, f32, vp, i32, vp, sz, vp, vp, vp, vp, vp, vp]
    L.zero_status_string.argtypes = [ctypes.c_int]
    L.zero_status_string.restype = ctypes.c_char_p
    L.zero_last_error.argtypes = []
    L.zero_last_error.restype = ctypes.c_char_p
    for nm in ("zero_shard_range", "zero_tensor_table", "zero_flatten_cast", "zero_accum", "zero_reduce_chunks",
               "zero_grad_sqnorm",
               "zero_grad_sqnorm_finalize", "zero_grad_sqnorm_combine", "zero_grad_sqnorm_noalloc",
               "zero_adamw_step", "zero_adamw_step_tensors", "zero_loss_scale_update", "zero_loss_scale_update_device",
               "zero_adamw_scalars",
               "zero_adamw_prepare_device", "zero_adamw_step_device", "zero_adamw_step_tensors_device",
               "zero_debug_errors", "zero_debug_selftest", "zero_state8_pack", "zero_state8_unpack",
               "zero_adamw_step8_tensors", "zero_adamw_step8_tensors_device", "zero_list_chunks", "zero_adamw_list",
               "zero_adamw_list_device", "zero_adamw_prepare_list_device", "zero_grad_plan", "zero_grad_entries_check",
               "zero_list_sums", "zero_sums_norms", "zero_list_clip", "zero_list_norms", "zero_adamw_list_clips",
               "zero_adamw_list_clips_device"):
        getattr(L, nm).restype = ctypes.c_int
    _lib = L
    return L


def _check(st: int) -> None:
    if st != ZERO_OK:
        L = lib()
        raise ZeroError(st, f"{L.zero_status_string(st).decode()}: {L.zero_last_error().decode()}")


def _dev(t: Optional[torch.Tensor], name: str, dtype=None, allow_none: bool = False):
    if t is None:
        if allow_none:
            return None
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _grad_ptr(t: torch.Tensor, name: str) -> int:
    """Address of a grad for the tensor table: a contiguous CUDA tensor, or a
    contiguous PINNED host tensor.  Pinned host memory is mapped into the
    device's unified address space at the same address, so the flatten
    kernel reads it directly over the host link (the host-to-device transfer
    and the flatten/cast become one pass).  Pageable host memory is refused."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.is_cuda:
        return t.data_ptr()
    if t.device.type == "cpu" and t.is_pinned():
        return t.data_ptr()
    raise ValueError(f"{name} must be a CUDA tensor or a pinned host tensor")


# the current stream's handle without a Stream object around it, where torch has that
_current_handle = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def _stream(stream) -> int:
    if type(stream) is int:
        return stream
    if stream is None:
        return _current_handle(torch.cuda.current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


# ------------------------------------------------------------------ host only
def zero_shard_range(total: int, world_size: int, rank: int) -> Tuple[int, int]:
    s, e = ctypes.c_int64(), ctypes.c_int64()
    _check(lib().zero_shard_range(total, world_size, rank, ctypes.byref(s), ctypes.byref(e)))
    return s.value, e.value


def zero_tensor_table(grads: Sequence[Optional[torch.Tensor]] = None, numels: Sequence[int] = None):
    """Host FlatParameter table for `grads` (None = no grad) or bare `numels`.

    Grads are CUDA tensors or pinned host tensors (read over the host link).
    Returns (table, total) where table is a ctypes array of zero_tensor.
    """
    if numels is None:
        numels = [0 if g is None else g.numel() for g in grads]
    n = len(numels)
    nm = np.ascontiguousarray(np.asarray(numels, dtype=np.int64))
    ptrs = None
    if grads is not None:
        ptrs = (ctypes.c_void_p * n)(*[None if g is None else _grad_ptr(g, f"grads[{i}]") for i, g in enumerate(grads)])
    table = (zero_tensor * max(n, 1))()
    total = ctypes.c_int64()
    _check(lib().zero_tensor_table(ptrs, ctypes.c_void_p(nm.ctypes.data), n, table, ctypes.byref(total)))
    return table, total.value


def device_table(table, n_tensors: int, device) -> torch.Tensor:
    """Copy a host table (from zero_tensor_table) into device memory (uint8 bytes)."""
    raw = bytes(memoryview(table))[: n_tensors * TENSOR_ENTRY_BYTES]
    host = torch.frombuffer(bytearray(raw), dtype=torch.uint8) if raw else torch.empty(0, dtype=torch.uint8)
    return host.to(device)


def zero_grad_sqnorm_workspace_bytes(n: int) -> int:
    return int(lib().zero_grad_sqnorm_workspace_bytes(n))


# --------------------------------------------------------------------- device
def _ws_bytes(ws: Optional[torch.Tensor]) -> int:
    return 0 if ws is None else ws.numel() * ws.element_size()


def _dscale(d_scale: Optional[torch.Tensor]):
    """A device float the kernels read their scale from (e.g. DeviceLossScale.unscale), or None."""
    if d_scale is None:
        return None
    if d_scale.dtype != torch.float32 or d_scale.numel() < 1:
        raise ValueError("d_scale must be a float32 device tensor")
    return _dev(d_scale, "d_scale")


# zero_flatten_cast's accumulate == 2: the norm of the accumulated sum only (nothing stored)
NORM_OF_SUM = 2


def _accum_mode(accumulate) -> int:
    if isinstance(accumulate, bool) or accumulate in (0, 1):
        return int(bool(accumulate))
    if accumulate == NORM_OF_SUM:
        return NORM_OF_SUM
    raise ValueError("accumulate must be False, True or NORM_OF_SUM")


def _check_acc(acc: Optional[torch.Tensor], n: int) -> None:
    if acc is not None and (acc.numel() != n or acc.dtype != torch.float32):
        raise ValueError("acc must be fp32 with master's size")


def zero_flatten_cast(d_table: torch.Tensor, n_tensors: int, total: int, src_dtype: torch.dtype, shard_start: int,
                      shard_end: int, scale: float, accumulate, dst: torch.Tensor,
                      found_nonfinite: Optional[torch.Tensor] = None, norm_ws: Optional[torch.Tensor] = None,
                      stream=None, d_scale: Optional[torch.Tensor] = None) -> None:
    """accumulate: False / True, or NORM_OF_SUM (2): the norm partials of dst + scale * x
    into norm_ws, dst only read."""
    if dst is not None and shard_end > shard_start and dst.numel() < shard_end - shard_start:
        raise ValueError("dst is smaller than the shard")
    tab = _dev(d_table, "d_table", torch.uint8, allow_none=n_tensors == 0)
    if n_tensors > 0 and d_table.numel() < n_tensors * TENSOR_ENTRY_BYTES:
        raise ValueError("d_table holds fewer entries than n_tensors")
    _check(lib().zero_flatten_cast(tab, n_tensors, total, _DT[src_dtype], shard_start, shard_end, scale,
                                   _dscale(d_scale), _accum_mode(accumulate),
                                   _dev(dst, "dst", torch.float32, allow_none=norm_ws is not None),
                                   _dev(found_nonfinite, "found_nonfinite", torch.int32, allow_none=True),
                                   _dev(norm_ws, "norm_ws", allow_none=True), _ws_bytes(norm_ws), _stream(stream)))


def zero_accum(acc: torch.Tensor, src: torch.Tensor, scale: float, accumulate: bool,
               found_nonfinite: Optional[torch.Tensor] = None, norm_ws: Optional[torch.Tensor] = None,
               stream=None, d_scale: Optional[torch.Tensor] = None) -> None:
    if src.numel() != acc.numel():
        raise ValueError("acc and src differ in size")
    _check(lib().zero_accum(_dev(acc, "acc", torch.float32), _dev(src, "src"), _DT[src.dtype], acc.numel(), scale,
                            _dscale(d_scale), int(bool(accumulate)),
                            _dev(found_nonfinite, "found_nonfinite", torch.int32, allow_none=True),
                            _dev(norm_ws, "norm_ws", allow_none=True), _ws_bytes(norm_ws), _stream(stream)))


def zero_reduce_chunks(acc: torch.Tensor, chunks: torch.Tensor, n: int, scale: float, accumulate: bool,
                       found_nonfinite: Optional[torch.Tensor] = None, norm_ws: Optional[torch.Tensor] = None,
                       stream=None, d_scale: Optional[torch.Tensor] = None) -> None:
    """acc[0:n] (+)= the rank-order sum of scale * chunks[r, 0:n] (chunks: a 2-D
    [n_chunks, chunk_stride] CUDA tensor of the received blocks, rank r's in row r)."""
    if chunks.dim() != 2:
        raise ValueError("chunks must be 2-D: [n_chunks, chunk_stride]")
    if chunks.dtype not in _DT:
        raise ValueError(f"chunks dtype {chunks.dtype} is not f32/bf16/f16")
    if acc.numel() < n or chunks.shape[1] < n:
        raise ValueError("acc or a chunk is shorter than n")
    _check(lib().zero_reduce_chunks(_dev(acc, "acc", torch.float32), _dev(chunks, "chunks"), _DT[chunks.dtype],
                                    chunks.shape[0], chunks.shape[1], n, scale, _dscale(d_scale),
                                    int(bool(accumulate)),
                                    _dev(found_nonfinite, "found_nonfinite", torch.int32, allow_none=True),
                                    _dev(norm_ws, "norm_ws", allow_none=True), _ws_bytes(norm_ws), _stream(stream)))


def zero_grad_sqnorm_finalize(ws: Optional[torch.Tensor], n: int, extra_sqnorm: float, max_norm: float,
                              out: torch.Tensor, stream=None) -> None:
    """Norm result from the partials a fused flatten/accumulate pass wrote for an n-element grad."""
    if out.numel() * out.element_size() < NORM_RESULT_BYTES:
        raise ValueError("out is smaller than zero_norm_result")
    if n > 0 and _ws_bytes(ws) < zero_grad_sqnorm_workspace_bytes(n):
        raise ValueError("ws is smaller than the partials of n elements")
    _check(lib().zero_grad_sqnorm_finalize(_dev(ws, "ws", allow_none=True), n, extra_sqnorm, max_norm,
                                           _dev(out, "out"), _stream(stream)))


def zero_grad_sqnorm(grad: torch.Tensor, extra_sqnorm: float, max_norm: float, ws: torch.Tensor,
                     out: torch.Tensor, stream=None) -> None:
    if out.numel() * out.element_size() < NORM_RESULT_BYTES:
        raise ValueError("out is smaller than zero_norm_result")
    _check(lib().zero_grad_sqnorm(_dev(grad, "grad", torch.float32), grad.numel(), extra_sqnorm, max_norm,
                                  _dev(ws, "ws", allow_none=True), 0 if ws is None else ws.numel() * ws.element_size(),
                                  _dev(out, "out"), _stream(stream)))


def zero_grad_sqnorm_noalloc(grad: torch.Tensor, extra_sqnorm: float, max_norm: float, out: torch.Tensor,
                             stream=None) -> None:
    """zero_grad_sqnorm for callers that cannot allocate a workspace (library-owned scratch)."""
    if out.numel() * out.element_size() < NORM_RESULT_BYTES:
        raise ValueError("out is smaller than zero_norm_result")
    _check(lib().zero_grad_sqnorm_noalloc(_dev(grad, "grad", torch.float32), grad.numel(), extra_sqnorm, max_norm,
                                          _dev(out, "out"), _stream(stream)))


def zero_grad_sqnorm_combine(sqnorms: torch.Tensor, max_norm: float, out: torch.Tensor, stream=None) -> None:
    """Global norm result from the ranks' local sums of squares (float64 CUDA vector, rank order)."""
    if out.numel() * out.element_size() < NORM_RESULT_BYTES:
        raise ValueError("out is smaller than zero_norm_result")
    _check(lib().zero_grad_sqnorm_combine(_dev(sqnorms, "sqnorms", torch.float64), sqnorms.numel(), max_norm,
                                          _dev(out, "out"), _stream(stream)))


def sqnorm_view(result: torch.Tensor) -> torch.Tensor:
    """The `sqnorm` field of a device zero_norm_result buffer as a 1-element float64 tensor view."""
    return result[:8].view(torch.float64)


def zero_adamw_step(master: torch.Tensor, exp_avg: torch.Tensor, exp_avg_sq: torch.Tensor, grad: torch.Tensor,
                    param_lowp: Optional[torch.Tensor], lr: float, beta1: float, beta2: float, eps: float,
                    weight_decay: float, step: int, clip: Optional[torch.Tensor] = None, stream=None) -> None:
    n = master.numel()
    for t, nm in ((exp_avg, "exp_avg"), (exp_avg_sq, "exp_avg_sq"), (grad, "grad")):
        if t.numel() != n:
            raise ValueError(f"{nm} differs in size from master")
    lowp_dt = ZERO_BF16
    if param_lowp is not None:
        if param_lowp.numel() != n:
            raise ValueError("param_lowp differs in size from master")
        if param_lowp.dtype not in (torch.bfloat16, torch.float16):
            raise ValueError("param_lowp must be bf16 or f16")
        lowp_dt = _DT[param_lowp.dtype]
    if clip is not None and clip.numel() * clip.element_size() < NORM_RESULT_BYTES:
        raise ValueError("clip is smaller than zero_norm_result")
    hp = zero_adamw_hparams(lr, beta1, beta2, eps, weight_decay)
    _check(lib().zero_adamw_step(_dev(master, "master", torch.float32), _dev(exp_avg, "exp_avg", torch.float32),
                                 _dev(exp_avg_sq, "exp_avg_sq", torch.float32), _dev(grad, "grad", torch.float32),
                                 _dev(param_lowp, "param_lowp", allow_none=True), lowp_dt, n, ctypes.byref(hp), step,
                                 _dev(clip, "clip", allow_none=True), _stream(stream)))


def zero_adamw_step_tensors(master: torch.Tensor, exp_avg: torch.Tensor, exp_avg_sq: torch.Tensor,
                            d_table: torch.Tensor, n_tensors: int, total: int, grad_dtype: torch.dtype,
                            shard_start: int, grad_scale: float, param_lowp: Optional[torch.Tensor], lr: float,
                            beta1: float, beta2: float, eps: float, weight_decay: float, step: int,
                            clip: Optional[torch.Tensor] = None, stream=None, acc: Optional[torch.Tensor] = None,
                            d_scale: Optional[torch.Tensor] = None) -> None:
    """AdamW over [shard_start, shard_start + n) with the grads read through the tensor table;
    acc: the earlier micro-batches' fp32 sum over the same n elements, added first (or None);
    d_scale: a device float used in place of grad_scale (or None)."""
    n = master.numel()
    for t, nm in ((exp_avg, "exp_avg"), (exp_avg_sq, "exp_avg_sq")):
        if t.numel() != n:
            raise ValueError(f"{nm} differs in size from master")
    _check_acc(acc, n)
    if n_tensors > 0 and d_table.numel() < n_tensors * TENSOR_ENTRY_BYTES:
        raise ValueError("d_table holds fewer entries than n_tensors")
    lowp_dt = ZERO_BF16
    if param_lowp is not None:
        if param_lowp.numel() != n or param_lowp.dtype not in (torch.bfloat16, torch.float16):
            raise ValueError("param_lowp must be bf16/f16 with master's size")
        lowp_dt = _DT[param_lowp.dtype]
    if clip is not None and clip.numel() * clip.element_size() < NORM_RESULT_BYTES:
        raise ValueError("clip is smaller than zero_norm_result")
    hp = zero_adamw_hparams(lr, beta1, beta2, eps, weight_decay)
    _check(lib().zero_adamw_step_tensors(_dev(master, "master", torch.float32), _dev(exp_avg, "exp_avg", torch.float32),
                                         _dev(exp_avg_sq, "exp_avg_sq", torch.float32),
                                         _dev(d_table, "d_table", torch.uint8, allow_none=n_tensors == 0), n_tensors,
                                         total, _DT[grad_dtype], shard_start, grad_scale, _dscale(d_scale),
                                         _dev(acc, "acc", torch.float32, allow_none=True),
                                         _dev(param_lowp, "param_lowp", allow_none=True), lowp_dt, n, ctypes.byref(hp),
                                         step, _dev(clip, "clip", allow_none=True), _stream(stream)))


# ------------------------------------------------- graph-capturable steps
def zero_adamw_scalars(lr: float, beta1: float, beta2: float, eps: float, weight_decay: float, step: int) -> np.ndarray:
    """The 8 binary32 scalars of step `step` (host): step_size, sqrt(1-beta2^t), 1-lr*wd,
    beta1, 1-beta1, beta2, 1-beta2, eps."""
    out = np.zeros(8, dtype=np.float32)
    hp = zero_adamw_hparams(lr, beta1, beta2, eps, weight_decay)
    _check(lib().zero_adamw_scalars(ctypes.byref(hp), step, ctypes.c_void_p(out.ctypes.data)))
    return out


def device_hparams(lr: float, beta1: float, beta2: float, eps: float, weight_decay: float, device,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """A zero_adamw_hparams in device memory (uint8 bytes); rewrites `out` in place when given."""
    hp = zero_adamw_hparams(lr, beta1, beta2, eps, weight_decay)
    host = torch.frombuffer(bytearray(bytes(memoryview(hp))), dtype=torch.uint8)
    if out is None:
        return host.to(device)
    out.copy_(host)
    return out


def new_adamw_device_state(device, step: int = 0) -> torch.Tensor:
    """Device buffer for one zero_adamw_device_state with the step count set (0: fresh)."""
    st = zero_adamw_device_state(step, 0, 0)
    return torch.frombuffer(bytearray(bytes(memoryview(st))), dtype=torch.uint8).to(device)


class AdamwDeviceState(NamedTuple):
    step: int
    apply: bool
    status: int
    scalars: np.ndarray


def decode_adamw_device_state(buf: torch.Tensor) -> AdamwDeviceState:
    raw = bytes(buf.detach().cpu().numpy().tobytes()[:DEVICE_STATE_BYTES])
    r = zero_adamw_device_state.from_buffer_copy(raw)
    return AdamwDeviceState(r.step, bool(r.apply), r.status, np.array(list(r.scalars), dtype=np.float32))


def _state_arg(state: torch.Tensor):
    if state.numel() * state.element_size() < DEVICE_STATE_BYTES:
        raise ValueError("state is smaller than zero_adamw_device_state")
    return _dev(state, "state")


def zero_adamw_prepare_device(d_hp: torch.Tensor, clip: Optional[torch.Tensor], state: torch.Tensor,
                              stream=None) -> None:
    """Advance the device step state for the next step (skipped on a non-finite norm)."""
    if d_hp.numel() * d_hp.element_size() < HPARAMS_BYTES:
        raise ValueError("d_hp is smaller than zero_adamw_hparams")
    if clip is not None and clip.numel() * clip.element_size() < NORM_RESULT_BYTES:
        raise ValueError("clip is smaller than zero_norm_result")
    _check(lib().zero_adamw_prepare_device(_dev(d_hp, "d_hp"), _dev(clip, "clip", allow_none=True),
                                           _state_arg(state), _stream(stream)))


def _lowp_arg(param_lowp: Optional[torch.Tensor], n: int):
    if param_lowp is None:
        return None, ZERO_BF16
    if param_lowp.numel() != n or param_lowp.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("param_lowp must be bf16/f16 with master's size")
    return _dev(param_lowp, "param_lowp"), _DT[param_lowp.dtype]


def zero_adamw_step_device(master: torch.Tensor, exp_avg: torch.Tensor, exp_avg_sq: torch.Tensor,
                           grad: torch.Tensor, param_lowp: Optional[torch.Tensor], state: torch.Tensor,
                           clip: Optional[torch.Tensor] = None, stream=None) -> None:
    """zero_adamw_step with the scalars and skip decision of the device step state."""
    n = master.numel()
    for t, nm in ((exp_avg, "exp_avg"), (exp_avg_sq, "exp_avg_sq"), (grad, "grad")):
        if t.numel() != n:
            raise ValueError(f"{nm} differs in size from master")
    if clip is not None and clip.numel() * clip.element_size() < NORM_RESULT_BYTES:
        raise ValueError("clip is smaller than zero_norm_result")
    lp, lowp_dt = _lowp_arg(param_lowp, n)
    _check(lib().zero_adamw_step_device(_dev(master, "master", torch.float32), _dev(exp_avg, "exp_avg", torch.float32),
                                        _dev(exp_avg_sq, "exp_avg_sq", torch.float32),
                                        _dev(grad, "grad", torch.float32), lp, lowp_dt, n, _state_arg(state),
                                        _dev(clip, "clip", allow_none=True), _stream(stream)))


def zero_adamw_step_tensors_device(master: torch.Tensor, exp_avg: torch.Tensor, exp_avg_sq: torch.Tensor,
                                   d_table: torch.Tensor, n_tensors: int, total: int, grad_dtype: torch.dtype,
                                   shard_start: int, grad_scale: float, param_lowp: Optional[torch.Tensor],
                                   state: torch.Tensor, clip: Optional[torch.Tensor] = None, stream=None,
                                   acc: Optional[torch.Tensor] = None, d_scale: Optional[torch.Tensor] = None) -> None:
    """zero_adamw_step_tensors with the scalars and skip decision of the device step state."""
    n = master.numel()
    for t, nm in ((exp_avg, "exp_avg"), (exp_avg_sq, "exp_avg_sq")):
        if t.numel() != n:
            raise ValueError(f"{nm} differs in size from master")
    _check_acc(acc, n)
    if n_tensors > 0 and d_table.numel() < n_tensors * TENSOR_ENTRY_BYTES:
        raise ValueError("d_table holds fewer entries than n_tensors")
    if clip is not None and clip.numel() * clip.element_size() < NORM_RESULT_BYTES:
        raise ValueError("clip is smaller than zero_norm_result")
    lp, lowp_dt = _lowp_arg(param_lowp, n)
    _check(lib().zero_adamw_step_tensors_device(
        _dev(master, "master", torch.float32), _dev(exp_avg, "exp_avg", torch.float32),
        _dev(exp_avg_sq, "exp_avg_sq", torch.float32), _dev(d_table, "d_table", torch.uint8, allow_none=n_tensors == 0),
        n_tensors, total, _DT[grad_dtype], shard_start, grad_scale, _dscale(d_scale),
        _dev(acc, "acc", torch.float32, allow_none=True), lp, lowp_dt, n, _state_arg(state),
        _dev(clip, "clip", allow_none=True), _stream(stream)))


# ------------------------------------------------- 8-bit moments, tensor lists
class State8(NamedTuple):
    """The 8-bit moments of n elements: e4m3 codes (float8_e4m3fn, n) of exp_avg and of the
    square root of exp_avg_sq, each with one fp32 power-of-two scale per 256 elements.
    exp_avg = code x scale; exp_avg_sq = (code x scale)^2."""
    exp_avg: torch.Tensor
    exp_avg_scale: torch.Tensor
    root: torch.Tensor
    root_scale: torch.Tensor


def state8_blocks(n: int) -> int:
    """Scales of n elements: ceil(n / 256)."""
    return -(-n // STATE8_BLOCK)


def new_state8(n: int, device) -> State8:
    """8-bit moments of n elements, all zero."""
    b = state8_blocks(n)
    codes = [torch.zeros(n, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.zeros(b, dtype=torch.float32, device=device) for _ in range(2)]
    return State8(codes[0], scales[0], codes[1], scales[1])


def _state8_arg(state: State8, n: int, who: str = "state8") -> zero_state8:
    if not isinstance(state, tuple) or len(state) != 4:
        raise ValueError(f"{who} must be a State8")
    m, ms, r, rs = state
    q = zero_state8(_dev(m, f"{who}.exp_avg", torch.float8_e4m3fn), _dev(ms, f"{who}.exp_avg_scale", torch.float32),
                    _dev(r, f"{who}.root", torch.float8_e4m3fn), _dev(rs, f"{who}.root_scale", torch.float32))
    b = -(-n // STATE8_BLOCK)
    if m.numel() != n or r.numel() != n or ms.numel() != b or rs.numel() != b:
        for t, nm, k in zip(state, State8._fields, (n, b, n, b)):
            if t.numel() != k:
                raise ValueError(f"{who}.{nm} has {t.numel()} elements, expected {k}")
    return q


DEFAULT_SEED = "default"


def rounding_choice(state_bits: int, rounding_seed):
    """The rounding_seed that an optimizer keeps: stochastic rounding with seed 0 unless told
    otherwise (8 bits), None with 32."""
    if state_bits not in (8, 32):
        raise ValueError("state_bits must be 32 or 8")
    if isinstance(rounding_seed, str):
        if rounding_seed != DEFAULT_SEED:
            raise ValueError("rounding_seed must be an integer or None")
        return 0 if state_bits == 8 else None
    if rounding_seed is not None and state_bits == 32:
        raise ValueError("a rounding_seed needs state_bits=8")
    return rounding_seed


def _rounding(rounding_seed: Optional[int], stream: int, root_bits: int):
    """NULL (round to nearest) or the 64-bit seed, the stream and the root's bits of stochastic rounding."""
    if rounding_seed is None:
        return None
    return ctypes.byref(zero_rounding(int(rounding_seed) & 0xFFFFFFFFFFFFFFFF, int(stream), int(root_bits), 0))


def zero_state8_pack(exp_avg: torch.Tensor, exp_avg_sq: torch.Tensor, state8: State8, stream=None) -> None:
    """fp32 moments into the 8-bit state, rounded to nearest."""
    n = exp_avg.numel()
    if exp_avg_sq.numel() != n:
        raise ValueError("exp_avg_sq differs in size from exp_avg")
    q = _state8_arg(state8, n)
    _check(lib().zero_state8_pack(_dev(exp_avg, "exp_avg", torch.float32),
                                  _dev(exp_avg_sq, "exp_avg_sq", torch.float32), n, ctypes.byref(q), _stream(stream)))


def zero_state8_unpack(state8: State8, exp_avg: torch.Tensor, exp_avg_sq: torch.Tensor, stream=None) -> None:
    """The fp32 moments that the 8-bit state stands for."""
    n = exp_avg.numel()
    if exp_avg_sq.numel() != n:
        raise ValueError("exp_avg_sq differs in size from exp_avg")
    q = _state8_arg(state8, n)
    _check(lib().zero_state8_unpack(ctypes.byref(q), n, _dev(exp_avg, "exp_avg", torch.float32),
                                    _dev(exp_avg_sq, "exp_avg_sq", torch.float32), _stream(stream)))


def check_moments(sd: dict, n: int) -> None:
    """Refuse a checkpoint whose moments are missing or not those of n elements."""
    saved = sd.get("state8")
    if saved is None:
        names, got, want = ("exp_avg", "exp_avg_sq"), (sd.get("exp_avg"), sd.get("exp_avg_sq")), (n, n)
    else:
        b = state8_blocks(n)
        names, got, want = State8._fields, tuple(saved), (n, b, n, b)
    if len(got) != len(want):
        raise ValueError("state8 of a checkpoint has four tensors")
    for nm, t, k in zip(names, got, want):
        if t is None or t.numel() != k:
            raise ValueError(f"the checkpoint's {nm} does not have the {k} elements expected")


def load_moments(sd: dict, state8: Optional[State8], exp_avg: Optional[torch.Tensor],
                 exp_avg_sq: Optional[torch.Tensor], device) -> None:
    """Copy a checkpoint's moments (fp32 exp_avg / exp_avg_sq, or state8) into an optimizer's,
    converting where the widths differ, on the current stream."""
    saved = sd.get("state8")
    if saved is None and state8 is None:
        exp_avg.copy_(sd["exp_avg"])
        exp_avg_sq.copy_(sd["exp_avg_sq"])
    elif saved is None:
        zero_state8_pack(sd["exp_avg"].to(device), sd["exp_avg_sq"].to(device), state8)
    elif state8 is None:
        zero_state8_unpack(State8(*(x.to(device) for x in saved)), exp_avg, exp_avg_sq)
    else:
        for dst, src in zip(state8, saved):
            dst.copy_(src)


def _step8_common(master, state8, d_table, n_tensors, param_lowp, clip, acc):
    n = master.numel()
    q = _state8_arg(state8, n)
    _check_acc(acc, n)
    if n_tensors > 0 and d_table.numel() < n_tensors * TENSOR_ENTRY_BYTES:
        raise ValueError("d_table holds fewer entries than n_tensors")
    if clip is not None and clip.numel() * clip.element_size() < NORM_RESULT_BYTES:
        raise ValueError("clip is smaller than zero_norm_result")
    lp, lowp_dt = _lowp_arg(param_lowp, n)
    return n, q, lp, lowp_dt


def zero_adamw_step8_tensors(master: torch.Tensor, state8: State8, d_table: torch.Tensor, n_tensors: int, total: int,
                             grad_dtype: torch.dtype, shard_start: int, grad_scale: float,
                             param_lowp: Optional[torch.Tensor], lr: float, beta1: float, beta2: float, eps: float,
                             weight_decay: float, step: int, clip: Optional[torch.Tensor] = None, stream=None,
                             acc: Optional[torch.Tensor] = None, d_scale: Optional[torch.Tensor] = None,
                             rounding_seed: Optional[int] = None, rounding_stream: Optional[int] = None,
                             root_bits: int = 0) -> None:
    """zero_adamw_step_tensors with the moments in 8 bits; rounding_seed: None rounds them to
    nearest, an integer seeds stochastic rounding, whose stream is rounding_stream (default:
    shard_start).  root_bits: the bits drawn for a root, 7 or 16; 0: 7 up to beta2 = 0.99,
    above it 16 (exp_avg: 7 up to beta1 = 0.95)."""
    n, q, lp, lowp_dt = _step8_common(master, state8, d_table, n_tensors, param_lowp, clip, acc)
    hp = zero_adamw_hparams(lr, beta1, beta2, eps, weight_decay)
    _check(lib().zero_adamw_step8_tensors(
        _dev(master, "master", torch.float32), ctypes.byref(q),
        _dev(d_table, "d_table", torch.uint8, allow_none=n_tensors == 0), n_tensors, total, _DT[grad_dtype],
        shard_start, grad_scale, _dscale(d_scale), _dev(acc, "acc", torch.float32, allow_none=True), lp, lowp_dt, n,
        ctypes.byref(hp), step, _rounding(rounding_seed, shard_start if rounding_stream is None else rounding_stream, root_bits),
        _dev(clip, "clip", allow_none=True), _stream(stream)))


def zero_adamw_step8_tensors_device(master: torch.Tensor, state8: State8, d_table: torch.Tensor, n_tensors: int,
                                    total: int, grad_dtype: torch.dtype, shard_start: int, grad_scale: float,
                                    param_lowp: Optional[torch.Tensor], state: torch.Tensor,
                                    clip: Optional[torch.Tensor] = None, stream=None,
                                    acc: Optional[torch.Tensor] = None, d_scale: Optional[torch.Tensor] = None,
                                    rounding_seed: Optional[int] = None, rounding_stream: Optional[int] = None,
                                    root_bits: int = 0) -> None:
    """zero_adamw_step8_tensors with the scalars, step and skip decision of the device step state."""
    n, q, lp, lowp_dt = _step8_common(master, state8, d_table, n_tensors, param_lowp, clip, acc)
    _check(lib().zero_adamw_step8_tensors_device(
        _dev(master, "master", torch.float32), ctypes.byref(q),
        _dev(d_table, "d_table", torch.uint8, allow_none=n_tensors == 0), n_tensors, total, _DT[grad_dtype],
        shard_start, grad_scale, _dscale(d_scale), _dev(acc, "acc", torch.float32, allow_none=True), lp, lowp_dt, n,
        _state_arg(state), _rounding(rounding_seed, shard_start if rounding_stream is None else rounding_stream, root_bits),
        _dev(clip, "clip", allow_none=True), _stream(stream)))


class TensorList(NamedTuple):
    """A list of tensors prepared for zero_adamw_list: the device copies of its entries and
    of the tensors' first chunks.  It holds addresses: keep the tensors alive."""
    entries: torch.Tensor      # uint8, 64 bytes per tensor
    first_chunk: torch.Tensor  # int32, one per tensor and their count
    n_chunks: int
    numels: Tuple[int, ...]
    state_bits: int
    n_groups: int
    lowp_dtype: Optional[torch.dtype]
    head: tuple                # the C entries' arguments that describe the list


_LIST_ENTRY = np.dtype([(nm, np.uint64 if ct is ctypes.c_void_p else np.int64 if ct is ctypes.c_int64 else np.int32)
                        for nm, ct in zero_list_tensor._fields_])


def make_tensor_list(columns: dict, numels: Sequence[int], group_of: Optional[Sequence[int]], n_groups: int,
                     state_bits: int, lowp_dtype: Optional[torch.dtype], device) -> TensorList:
    """Check a list given by columns of addresses (fields of zero_list_tensor; absent: NULL)
    and copy it to the device."""
    n = len(numels)
    entries = np.zeros(n, dtype=_LIST_ENTRY)
    for nm, col in columns.items():
        entries[nm] = col
    entries["numel"] = numels
    if group_of is not None:
        entries["group"] = group_of
    first = np.zeros(n + 1, dtype=np.int32)
    _check(lib().zero_list_chunks(entries.ctypes.data, n, n_groups, state_bits, first.ctypes.data, None))
    d_entries, d_first = torch.from_numpy(entries.view(np.uint8)).to(device), torch.from_numpy(first).to(device)
    head = (d_entries.data_ptr(), n, d_first.data_ptr(), int(first[-1]), state_bits)
    return TensorList(d_entries, d_first, int(first[-1]), tuple(numels), state_bits, n_groups, lowp_dtype, head)


def list_masters(masters: Sequence[torch.Tensor], lowp: Optional[Sequence[Optional[torch.Tensor]]],
                 group_of: Optional[Sequence[int]]):
    """The checked masters and copies of a list: (columns, numels, the copies' dtype)."""
    n = len(masters)
    if n == 0:
        raise ValueError("an empty tensor list")
    if (lowp is not None and len(lowp) != n) or (group_of is not None and len(group_of) != n):
        raise ValueError("masters, lowp and group_of differ in length")
    dev = masters[0].device
    ptrs, numels, copies, dts = [], [], [], set()
    for i, p in enumerate(masters):
        if not p.is_cuda or p.device != dev or p.dtype != torch.float32 or not p.is_contiguous():
            _dev(p, f"masters[{i}]", torch.float32)
            raise ValueError(f"masters[{i}] is not on one device with the list")
        ptrs.append(p.data_ptr())
        numels.append(p.numel())
    for i, c in enumerate(lowp or ()):
        if c is None:
            copies.append(0)
            continue
        copies.append(_dev(c, f"lowp[{i}]"))
        dts.add(c.dtype)
        if c.numel() != numels[i]:
            raise ValueError(f"lowp[{i}] differs in size from masters[{i}]")
        if c.device != dev:
            raise ValueError(f"lowp[{i}] is not on one device with the list")
    if len(dts) > 1 or not dts <= {torch.bfloat16, torch.float16}:
        raise ValueError("low-precision copies must be all bf16 or all f16")
    columns = {"master": ptrs}
    if lowp is not None:
        columns["lowp"] = copies
    return columns, numels, dts.pop() if dts else None


def zero_tensor_list(masters: Sequence[torch.Tensor], states: Sequence[tuple],
                     lowp: Optional[Sequence[Optional[torch.Tensor]]] = None, group_of: Optional[Sequence[int]] = None,
                     n_groups: int = 1, state_bits: int = 32) -> TensorList:
    """Check a list and copy it to the device.  states[i]: (exp_avg, exp_avg_sq), fp32, or
    with state_bits=8 a State8; lowp[i]: None or a bf16/f16 copy (one dtype for the list)."""
    if state_bits not in (8, 32):
        raise ValueError("state_bits must be 32 or 8")
    if len(states) != len(masters):
        raise ValueError("masters and states differ in length")
    columns, numels, lowp_dtype = list_masters(masters, lowp, group_of)
    moments = []
    for i, (st, k) in enumerate(zip(states, numels)):
        if any(t.device != masters[0].device for t in st):
            raise ValueError(f"states[{i}] is not on one device with the list")
        if state_bits == 8:
            q = _state8_arg(st, k, f"states[{i}]")
            moments.append((q.exp_avg or 0, q.root or 0, q.exp_avg_scale or 0, q.root_scale or 0))
        else:
            if len(st) != 2 or st[0].numel() != k or st[1].numel() != k:
                raise ValueError(f"states[{i}] differs in size from masters[{i}]")
            moments.append((_dev(st[0], f"states[{i}].exp_avg", torch.float32),
                            _dev(st[1], f"states[{i}].exp_avg_sq", torch.float32)))
    for nm, col in zip(("exp_avg", "exp_avg_sq", "exp_avg_scale", "root_scale"), zip(*moments)):
        columns[nm] = col
    return make_tensor_list(columns, numels, group_of, n_groups, state_bits, lowp_dtype, masters[0].device)


def _list_args(tl: TensorList, d_grads: torch.Tensor, grad_dtype: torch.dtype, grad_scale: float, d_scale):
    if d_grads.numel() < len(tl.numels) * TENSOR_ENTRY_BYTES:
        raise ValueError("d_grads holds fewer entries than the list")
    return (*tl.head, _dev(d_grads, "d_grads", torch.uint8), _DT[grad_dtype], grad_scale,
            None if d_scale is None else _dscale(d_scale), ZERO_BF16 if tl.lowp_dtype is None else _DT[tl.lowp_dtype])


def list_groups(groups: Sequence[Tuple[float, float, float, float, float]]):
    """(lr, beta1, beta2, eps, weight_decay) of each group as zero_adamw_list takes them."""
    return (zero_adamw_hparams * len(groups))(*[zero_adamw_hparams(*g) for g in groups])


def _check_clip(tl: TensorList, clip: Optional[torch.Tensor], clips: bool) -> None:
    need = (tl.n_groups + 1 if clips else 1) * NORM_RESULT_BYTES
    if clips and clip is None:
        raise ValueError("clips needs the groups' results")
    if clip is not None and clip.numel() * clip.element_size() < need:
        raise ValueError("clip is smaller than one zero_norm_result per group and one more" if clips
                         else "clip is smaller than zero_norm_result")


def zero_adamw_list(tl: TensorList, d_grads: torch.Tensor, grad_dtype: torch.dtype, grad_scale: float,
                    groups: Sequence[Tuple[float, float, float, float, float]], step: int,
                    clip: Optional[torch.Tensor] = None, stream=None, d_scale: Optional[torch.Tensor] = None,
                    rounding_seed: Optional[int] = None, rounding_stream: int = 0, root_bits: int = 0,
                    clips: bool = False) -> None:
    """One AdamW step over every tensor of a list.  d_grads: the device table of the grads
    (zero_tensor_table + device_table, in list order); groups: (lr, beta1, beta2, eps,
    weight_decay) of each parameter group, or list_groups() of them made once.  rounding_seed,
    root_bits: as for zero_adamw_step8_tensors (each tensor by its group's beta2).  clips: clip
    holds a result for each group and one over all (GradClip.results), not one."""
    if len(groups) != tl.n_groups:
        raise ValueError(f"{len(groups)} groups given, the list has {tl.n_groups}")
    _check_clip(tl, clip, clips)
    hp = groups if isinstance(groups, ctypes.Array) else list_groups(groups)
    call = lib().zero_adamw_list_clips if clips else lib().zero_adamw_list
    _check(call(*_list_args(tl, d_grads, grad_dtype, grad_scale, d_scale), hp, len(groups), step,
                _rounding(rounding_seed, rounding_stream, root_bits), _dev(clip, "clip", allow_none=True),
                _stream(stream)))


def zero_adamw_list_device(tl: TensorList, d_grads: torch.Tensor, grad_dtype: torch.dtype, grad_scale: float,
                           states: torch.Tensor, clip: Optional[torch.Tensor] = None, stream=None,
                           d_scale: Optional[torch.Tensor] = None, rounding_seed: Optional[int] = None,
                           rounding_stream: int = 0, root_bits: int = 0, clips: bool = False) -> None:
    """zero_adamw_list with the groups' scalars, step and skip decision from device step states."""
    if states.numel() * states.element_size() < tl.n_groups * DEVICE_STATE_BYTES:
        raise ValueError("states is smaller than one zero_adamw_device_state per group")
    _check_clip(tl, clip, clips)
    call = lib().zero_adamw_list_clips_device if clips else lib().zero_adamw_list_device
    _check(call(*_list_args(tl, d_grads, grad_dtype, grad_scale, d_scale), _dev(states, "states"), tl.n_groups,
                _rounding(rounding_seed, rounding_stream, root_bits), _dev(clip, "clip", allow_none=True),
                _stream(stream)))


def zero_adamw_prepare_list_device(d_hp: torch.Tensor, n_groups: int, clip: Optional[torch.Tensor],
                                   states: torch.Tensor, stream=None) -> None:
    """Advance every group's device step state for the next step (all or none)."""
    if d_hp.numel() * d_hp.element_size() < n_groups * HPARAMS_BYTES:
        raise ValueError("d_hp is smaller than one zero_adamw_hparams per group")
    if states.numel() * states.element_size() < n_groups * DEVICE_STATE_BYTES:
        raise ValueError("states is smaller than one zero_adamw_device_state per group")
    if clip is not None and clip.numel() * clip.element_size() < NORM_RESULT_BYTES:
        raise ValueError("clip is smaller than zero_norm_result")
    _check(lib().zero_adamw_prepare_list_device(_dev(d_hp, "d_hp"), n_groups, _dev(clip, "clip", allow_none=True),
                                                _dev(states, "states"), _stream(stream)))


# ------------------------------------------------- norms and clipping of a list
_NORM_TYPES = {math.inf: 0, 1.0: 1, 2.0: 2}


class GradList(NamedTuple):
    """A grads list prepared for zero_list_norms and the like: the device copies of its
    entries and plan.  It holds addresses: keep the tensors alive."""
    entries: Optional[torch.Tensor]  # uint8, 40 bytes per tensor; None: sums and norms of other ranks' lists only
    plan: "GradPlan"
    ref: object                      # a pointer to the C entries' description of the list


class GradPlan(NamedTuple):
    """The work split of a grads list (zero_grad_plan) on the device: by sizes and groups alone."""
    ints: torch.Tensor  # int32
    numels: np.ndarray  # int64
    groups: Optional[np.ndarray]  # int32, or None: all in group 0
    n_groups: int
    head: zero_grad_list  # the C entries' description of the plan


_GRAD_ENTRY = np.dtype([(nm, np.uint64 if ct is ctypes.c_void_p else np.int64 if ct is ctypes.c_int64 else np.int32)
                        for nm, ct in zero_grad_entry._fields_])


def _to_device(a: np.ndarray, device, wait: bool) -> torch.Tensor:
    """A copy on the device.  wait: done when this returns, so that any stream may read it; else
    in the order of the current stream, without waiting for what runs there."""
    t = torch.from_numpy(a)
    if wait or torch.device(device).type != "cuda":
        return t.to(device)
    return t.pin_memory().to(device, non_blocking=True)


def zero_grad_plan(numels: Sequence[int], group_of: Optional[Sequence[int]], n_groups: int, norm_type: float,
                   device, wait: bool = True) -> GradPlan:
    """The plan of a list with these sizes and groups (group_of None: all in group 0), copied to the
    device.  wait=False: for the current stream alone, here and in what follows."""
    p = _NORM_TYPES.get(float(norm_type))
    if p is None:
        raise ValueError(f"norm_type must be 1, 2 or inf, got {norm_type}")
    n = len(numels)
    sizes = np.ascontiguousarray(np.asarray(numels, dtype=np.int64))
    groups = None
    if group_of is not None:
        if len(group_of) != n:
            raise ValueError("one group per tensor is required")
        groups = np.ascontiguousarray(np.asarray(group_of, dtype=np.int32))
    ints = np.zeros(4 * n + max(int(n_groups), 0) + 2, dtype=np.int32)
    head = zero_grad_list()
    _check(lib().zero_grad_plan(sizes.ctypes.data, None if groups is None else groups.ctypes.data, n, n_groups,
                                ints.ctypes.data, ctypes.byref(head)))
    d_ints = _to_device(ints, device, wait)
    head.d_plan, head.norm_type = d_ints.data_ptr(), p
    return GradPlan(d_ints, sizes, groups, int(n_groups), head)


def _dense(t: torch.Tensor) -> bool:
    """Whether the elements fill one run of memory, each address once."""
    if t.is_contiguous():
        return True
    size = 1
    for stride, k in sorted((s, k) for s, k in zip(t.stride(), t.shape) if k != 1):
        if stride != size:
            return False
        size *= k
    return True


def _overlaps(starts: np.ndarray, ends: np.ndarray, written: np.ndarray) -> bool:
    """Whether an interval that is written overlaps any other one."""
    order = np.argsort(starts, kind="stable")
    s, e, w = starts[order], ends[order], written[order]
    reach = np.maximum.accumulate(e)  # how far the earlier ones go, and the written ones among them
    reach_w = np.maximum.accumulate(np.where(w, e, 0))
    return bool(np.any((s[1:] < reach[:-1]) & w[1:]) or np.any(s[1:] < reach_w[:-1]))


def _addresses_of(tensors: Sequence[Optional[torch.Tensor]], sizes: List[int], device: torch.device, name: str):
    """The checked tensors' addresses and types (0 for None)."""
    cuda, index = device.type == "cuda", device.index if device.type == "cuda" else -1
    ptrs, dts = [0] * len(sizes), [0] * len(sizes)
    for i, t in enumerate(tensors):
        if t is None:
            continue
        if not isinstance(t, torch.Tensor) or not (t.is_cuda if cuda else t.is_cpu) or t.get_device() != index:
            raise ValueError(f"{name}[{i}] must be a tensor on {device}")
        dt = _DT.get(t.dtype)
        if dt is None:
            raise ValueError(f"{name}[{i}] is {t.dtype}, not f32, bf16 or f16")
        if t.numel() != sizes[i]:
            raise ValueError(f"{name}[{i}] has {t.numel()} elements, expected {sizes[i]}")
        if not t.is_contiguous() and not _dense(t):
            raise ValueError(f"{name}[{i}] does not fill one run of memory (strides {t.stride()})")
        ptrs[i], dts[i] = t.data_ptr(), dt
        if ptrs[i] == 0 and sizes[i]:  # NULL would read as no grad
            raise ValueError(f"{name}[{i}] has no memory (its storage was freed)")
    return ptrs, dts


def grad_list(plan: GradPlan, grads: Sequence[Optional[torch.Tensor]], out: Optional[Sequence] = None,
              write: bool = True, wait: bool = True) -> GradList:
    """Check a list of grads (None: no grad, reads as zeros) and copy it to the device.  out:
    where the clipped grads go, per tensor a buffer or None (that tensor is not written);
    out=None with write: in place.  Every tensor is f32, bf16 or f16, fills one run
    of memory (any order of its dimensions; its out in the same order), and overlaps no
    other that is written.  The device is the plan's."""
    n = len(plan.numels)
    if len(grads) != n or (out is not None and len(out) != n):
        raise ValueError("one grad (or None) per tensor is required, and one out")
    device = plan.ints.device
    entries = np.zeros(n, dtype=_GRAD_ENTRY)
    sizes = plan.numels.tolist()
    src, sdt = _addresses_of(grads, sizes, device, "grads")
    if not write:
        dst, ddt = [0] * n, [0] * n
    elif out is None:
        dst, ddt = src, sdt
    else:
        dst, ddt = _addresses_of(out, sizes, device, "out")
        for i, (g, y) in enumerate(zip(grads, out)):
            if g is None or y is None or (g.is_contiguous() and y.is_contiguous()):
                continue
            if g.shape != y.shape or g.stride() != y.stride():
                raise ValueError(f"out[{i}] is not laid out as its grad")
    entries["src"], entries["dst"], entries["src_dtype"], entries["dst_dtype"] = src, dst, sdt, ddt
    return _checked_list(plan, entries, wait)


def flat_grad_list(plan: GradPlan, flat: torch.Tensor, starts: np.ndarray) -> GradList:
    """The list of a flat grad's pieces, clipped in place: tensor i's plan.numels[i] elements from starts[i]."""
    if flat.device != plan.ints.device or flat.dtype not in _DT or flat.dim() != 1 or not flat.is_contiguous():
        raise ValueError(f"the flat grad must be 1-D, contiguous, f32, bf16 or f16, on {plan.ints.device}")
    if flat.untyped_storage().nbytes() < (flat.storage_offset() + flat.numel()) * flat.element_size():
        raise ValueError("the flat grad has no memory (its storage was freed)")
    some = plan.numels > 0
    if np.any(some & ((starts < 0) | (starts + plan.numels > flat.numel()))):
        raise ValueError("a piece lies outside the flat grad")
    entries = np.zeros(len(plan.numels), dtype=_GRAD_ENTRY)
    entries["src"] = np.where(some, np.uint64(flat.data_ptr()) + np.where(some, starts, 0).astype(np.uint64) *
                              np.uint64(flat.element_size()), np.uint64(0))
    entries["dst"], entries["src_dtype"], entries["dst_dtype"] = entries["src"], _DT[flat.dtype], _DT[flat.dtype]
    return _checked_list(plan, entries)


def _checked_list(plan: GradPlan, entries: np.ndarray, wait: bool = True) -> GradList:
    entries["numel"] = plan.numels
    if plan.groups is not None:
        entries["group"] = plan.groups
    _check(lib().zero_grad_entries_check(entries.ctypes.data, plan.numels.ctypes.data, len(entries), plan.n_groups))
    written = (entries["dst"] != 0) & (plan.numels > 0)
    if written.any():
        bytes_of = np.array([4, 2, 2], dtype=np.uint64)
        size = plan.numels.astype(np.uint64)
        read = (entries["src"] != 0) & (plan.numels > 0) & (entries["src"] != entries["dst"])
        at = np.concatenate([entries["dst"][written], entries["src"][read]])
        ends = at + np.concatenate([(size * bytes_of[entries["dst_dtype"]])[written],
                                    (size * bytes_of[entries["src_dtype"]])[read]])
        if _overlaps(at, ends, np.arange(len(at)) < int(written.sum())):
            raise ValueError("a grad that is written overlaps another tensor of the list (is one listed twice?)")
    d_entries = _to_device(entries.view(np.uint8), plan.ints.device, wait)
    elsewhere = (entries["dst"] != 0) & (entries["dst"] != entries["src"])
    return GradList(d_entries, plan, _list_ref(plan, d_entries.data_ptr(), int(not elsewhere.any())))


def _list_ref(plan: GradPlan, d_entries: Optional[int], in_place: int):
    head = zero_grad_list.from_buffer_copy(plan.head)
    head.d_entries, head.in_place = d_entries, in_place
    return ctypes.pointer(head)


def norms_only_list(plan: GradPlan) -> GradList:
    """A list without entries, for zero_sums_norms."""
    return GradList(None, plan, _list_ref(plan, None, 0))


def zero_list_norms_workspace_bytes(plan: GradPlan) -> int:
    return int(lib().zero_list_norms_workspace_bytes(ctypes.byref(plan.head)))


class NormBuffers(NamedTuple):
    """What the calls on lists of one plan read and write, made by norm_buffers."""
    plan: GradPlan
    ws: torch.Tensor           # uint8, zero_list_norms_workspace_bytes
    sums: torch.Tensor         # float64, a tensor's sum each
    joined: torch.Tensor       # float64, the same over all ranks (zero_sums_norms)
    max_norms: torch.Tensor    # float64, the groups' limits (read)
    norms: torch.Tensor        # float32: tensors, groups, all
    results: torch.Tensor      # a zero_norm_result per group and one for all
    found: torch.Tensor        # int32, set where the norm over all is not finite
    addresses: Optional[tuple]  # ws, its bytes, sums, joined, max_norms, norms, results, found; None: host memory


def norm_buffers(plan: GradPlan, max_norms: torch.Tensor, wait: bool = True) -> NormBuffers:
    """Buffers for lists of this plan, zeros (wait=False: as a launch fills them); max_norms: the
    groups' limits (float64, on the device)."""
    dev, n, g = plan.ints.device, len(plan.numels), plan.n_groups
    if max_norms.dtype != torch.float64 or max_norms.numel() != g or max_norms.device != dev or not max_norms.is_contiguous():
        raise ValueError(f"max_norms must be {g} float64 on {dev}")
    ws = torch.empty(max(zero_list_norms_workspace_bytes(plan), 8), dtype=torch.uint8, device=dev)
    new = torch.zeros if wait else torch.empty
    sums, joined = (new(n, dtype=torch.float64, device=dev) for _ in range(2))
    norms = new(n + g + 1, dtype=torch.float32, device=dev)
    results = new((g + 1) * NORM_RESULT_BYTES, dtype=torch.uint8, device=dev)
    found = torch.zeros(1, dtype=torch.int32, device=dev)
    if wait and ws.is_cuda:  # the zeros are there before a launch on any stream
        torch.cuda.current_stream(dev).synchronize()
    addresses = (ws.data_ptr(), ws.numel(), sums.data_ptr(), joined.data_ptr(), max_norms.data_ptr(), norms.data_ptr(),
                 results.data_ptr(), found.data_ptr()) if ws.is_cuda else None
    return NormBuffers(plan, ws, sums, joined, max_norms, norms, results, found, addresses)


def _addresses(buffers: NormBuffers, gl: GradList, found: Optional[torch.Tensor] = None) -> tuple:
    """The buffers' addresses, which must be device memory and of this list's plan."""
    if buffers.plan is not gl.plan:
        raise ValueError("the buffers belong to another plan")
    if buffers.addresses is None:
        raise ValueError("the buffers must be CUDA tensors")
    if found is None:
        return buffers.addresses
    return buffers.addresses[:7] + (_dev(found, "found_nonfinite", torch.int32),)


def zero_list_sums(gl: GradList, scale: float, buffers: NormBuffers, stream=None,
                   d_scale: Optional[torch.Tensor] = None) -> None:
    """Each tensor's sum of |scale x|^p (the largest for p = inf) into buffers.sums."""
    a = _addresses(buffers, gl)
    _check(lib().zero_list_sums(gl.ref, scale, None if d_scale is None else _dscale(d_scale), a[0], a[1], a[2],
                                _stream(stream)))


def zero_sums_norms(gl: GradList, sums: torch.Tensor, n_parts: int, buffers: NormBuffers,
                    found_nonfinite: Optional[torch.Tensor] = None, stream=None) -> None:
    """The norms of tensors, groups and all from n_parts rows of sums, joined in row order.
    found_nonfinite: in place of the buffers' own."""
    _, _, _, joined, limits, norms, results, found = _addresses(buffers, gl, found_nonfinite)
    if sums.numel() < n_parts * len(gl.plan.numels):
        raise ValueError(f"sums has fewer than {n_parts} rows")
    _check(lib().zero_sums_norms(gl.ref, _dev(sums, "sums", torch.float64), n_parts, joined, limits, norms, results,
                                 found, _stream(stream)))


def zero_list_clip(gl: GradList, scale: float, buffers: NormBuffers, stream=None,
                   d_scale: Optional[torch.Tensor] = None) -> None:
    """Every tensor with a destination scaled and clipped by its group's coefficient in buffers.results."""
    _check(lib().zero_list_clip(gl.ref, scale, None if d_scale is None else _dscale(d_scale),
                                _addresses(buffers, gl)[6], _stream(stream)))


def zero_list_norms(gl: GradList, scale: float, clip: bool, buffers: NormBuffers,
                    found_nonfinite: Optional[torch.Tensor] = None, stream=None,
                    d_scale: Optional[torch.Tensor] = None) -> None:
    """zero_list_sums, zero_sums_norms of one part and, with clip, zero_list_clip in one call."""
    ws, nb, sums, _, limits, norms, results, found = _addresses(buffers, gl, found_nonfinite)
    _check(lib().zero_list_norms(gl.ref, scale, None if d_scale is None else _dscale(d_scale), clip, ws, nb, sums,
                                 limits, norms, results, found, _stream(stream)))


# ------------------------------------------------------------ debug builds
class DebugRecord(NamedTuple):
    count: int
    site: int
    index: int
    block: int


def zero_debug_errors(reset: bool = False) -> DebugRecord:
    """Access-check violations the debug library recorded (ZeroError on a release library)."""
    out = np.zeros(4, dtype=np.uint64)
    _check(lib().zero_debug_errors(ctypes.c_void_p(out.ctypes.data), int(bool(reset))))
    return DebugRecord(*(int(x) for x in out))


def zero_debug_selftest(index: int, stream=None) -> None:
    _check(lib().zero_debug_selftest(index, _stream(stream)))


# ------------------------------------------------------------ norm result I/O
class NormResult(NamedTuple):
    sqnorm: float
    norm: float
    clip_coef: float
    finite: bool


def new_norm_result(device) -> torch.Tensor:
    """Device buffer for one zero_norm_result (8-byte aligned by the allocator)."""
    return torch.zeros(NORM_RESULT_BYTES, dtype=torch.uint8, device=device)


def decode_norm_result(buf: torch.Tensor) -> NormResult:
    """Read a zero_norm_result (device or host bytes) into Python values."""
    raw = bytes(buf.detach().cpu().numpy().tobytes()[:NORM_RESULT_BYTES])
    r = zero_norm_result.from_buffer_copy(raw)
    return NormResult(r.sqnorm, r.norm, r.clip_coef, bool(r.finite))


# ------------------------------------------------------------ loss scaling
class DynamicLossScale:
    """GradScaler-style dynamic loss scale (host policy: zero_loss_scale_update).

    Multiply the loss by ``scale`` before backward; pass ``unscale_factor(accum_steps)``
    as the flatten / accumulate ``scale`` (the unscale and the 1/accum_steps
    averaging in one exact multiply for power-of-two values); after the step call
    ``update(found_inf)`` with the kernels' non-finite flag.
    """

    def __init__(self, init_scale: float = 2.0 ** 16, growth_factor: float = 2.0, backoff_factor: float = 0.5,
                 growth_interval: int = 2000):
        self._scale = ctypes.c_float(init_scale)
        self._good = ctypes.c_int32(0)
        self.growth_factor, self.backoff_factor, self.growth_interval = growth_factor, backoff_factor, growth_interval

    @property
    def scale(self) -> float:
        return self._scale.value

    @property
    def growth_tracker(self) -> int:
        return self._good.value

    def unscale_factor(self, accum_steps: int = 1) -> float:
        return 1.0 / (float(self._scale.value) * accum_steps)

    def update(self, found_inf: bool) -> None:
        _check(lib().zero_loss_scale_update(ctypes.byref(self._scale), ctypes.byref(self._good), int(bool(found_inf)),
                                            self.growth_factor, self.backoff_factor, self.growth_interval))


def zero_loss_scale_update_device(state: torch.Tensor, accum_steps: int, growth_factor: float,
                                  backoff_factor: float, growth_interval: int,
                                  norm_result: Optional[torch.Tensor] = None, stream=None) -> None:
    """The loss-scale update on a zero_loss_scale_state in device memory (one thread)."""
    if state.numel() * state.element_size() < LOSS_SCALE_STATE_BYTES:
        raise ValueError("state is smaller than zero_loss_scale_state")
    if norm_result is not None and norm_result.numel() * norm_result.element_size() < NORM_RESULT_BYTES:
        raise ValueError("norm_result is smaller than zero_norm_result")
    _check(lib().zero_loss_scale_update_device(_dev(state, "state"), accum_steps, growth_factor, backoff_factor,
                                               growth_interval, _dev(norm_result, "norm_result", allow_none=True),
                                               _stream(stream)))


class DeviceLossScale:
    """The GradScaler-style dynamic loss scale kept in device memory (a
    zero_loss_scale_state), for mixed-precision steps captured in a CUDA graph.

    The grad passes read ``unscale`` (= 1/(scale * accum_steps)) from device
    memory when they run (``d_scale``) and raise ``found_inf``
    (``found_nonfinite``); ``launch_update()`` (one thread, capturable) backs
    the scale off or grows it on the device, recomputes ``unscale`` and clears
    the flag.  The same rule and roundings as DynamicLossScale.update, so both
    follow the same scale bit for bit.  ``scale``, ``growth_tracker`` and
    ``read()`` copy the state to the host (a synchronisation)."""

    def __init__(self, device, init_scale: float = 2.0 ** 16, growth_factor: float = 2.0,
                 backoff_factor: float = 0.5, growth_interval: int = 2000, accum_steps: int = 1):
        if accum_steps < 1:
            raise ValueError("accum_steps must be >= 1")
        self.growth_factor, self.backoff_factor, self.growth_interval = growth_factor, backoff_factor, growth_interval
        self.accum_steps = int(accum_steps)
        sc = ctypes.c_float(init_scale).value
        st = zero_loss_scale_state(sc, 0, ctypes.c_float(1.0 / (float(sc) * self.accum_steps)).value, 0)
        self.state = torch.frombuffer(bytearray(bytes(memoryview(st))), dtype=torch.uint8).to(device)
        self.unscale = self.state[8:12].view(torch.float32)     # the grad passes' d_scale
        self.found_inf = self.state[12:16].view(torch.int32)    # the grad passes' found_nonfinite

    def launch_update(self, norm_result: Optional[torch.Tensor] = None, stream=None) -> None:
        """Enqueue the update after a step (norm_result: the step's zero_norm_result, whose
        non-finite norm also counts as an overflow)."""
        zero_loss_scale_update_device(self.state, self.accum_steps, self.growth_factor, self.backoff_factor,
                                      self.growth_interval, norm_result, stream)

    def read(self) -> zero_loss_scale_state:
        raw = bytes(self.state.detach().cpu().numpy().tobytes()[:LOSS_SCALE_STATE_BYTES])
        return zero_loss_scale_state.from_buffer_copy(raw)

    @property
    def scale(self) -> float:
        return self.read().scale

    @property
    def growth_tracker(self) -> int:
        return self.read().growth_tracker
