"""ctypes binding of libcutbce (include/cutbce.h): argument marshalling only.

Every step of the loss and its gradient runs in the library's CUDA kernels;
this module only turns torch tensors into pointers and sizes, takes the
current CUDA stream, and allocates outputs and the workspace through torch.
There is no CPU fallback: if the library is missing, importing a function that
needs it raises.
"""
from __future__ import annotations

import ctypes
import os
import re
from typing import Optional

import torch

__all__ = [
    "CutBCEError", "cutbce_problem", "load_library", "library_path", "declared_functions",
    "cutbce_workspace_size", "cutbce_workspace_size_for", "OUT_LOSS", "OUT_DH", "OUT_DE", "OUT_METRICS",
    "cutbce_options", "make_options", "cutbce_forward_backward_ex", "cutbce_workspace_size_ex",
    "GRAD_F32", "GRAD_BF16", "ACCUMULATE_DH", "ACCUMULATE_DE", "cutbce_forward", "cutbce_forward_fixed_scratch", "FIXED_SCRATCH_BYTES",
    "cutbce_backward", "cutbce_forward_backward",
    "cutbce_host_buffer_size", "cutbce_forward_backward_host", "cutbce_read_status",
    "cutbce_read_counts", "cutbce_kernel_launches", "cutbce_status_string",
    "cutbce_selftest_wait_timeout", "cutbce_selftest_element_math", "cutbce_topk_workspace_size", "cutbce_topk",
    "cutbce_hit_at_k", "cutbce_profile_enable", "cutbce_profile_read", "REDUCTIONS",
    "cutbce_grad_options", "cutbce_distill_problem", "cutbce_preference_problem", "make_distill_problem",
    "make_preference_problem", "cutbce_embed_forward", "cutbce_embed_workspace_size", "cutbce_embed_backward",
    "cutbce_distill_workspace_size", "cutbce_distill_forward", "cutbce_distill_backward",
    "cutbce_distill_forward_backward", "cutbce_preference_workspace_size", "cutbce_preference_forward",
    "cutbce_preference_backward", "cutbce_preference_forward_backward",
    "KERNEL_KINDS", "cutbce_probe_scratch_bytes", "cutbce_probe_pipe_rate", "PROBES", "cutbce_probe_mma",
]

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_TARGET_RANGE, ERR_TIMEOUT, ERR_CUDA = range(7)
BF16, F32 = 0, 1
OUT_LOSS, OUT_DH, OUT_DE, OUT_METRICS = 1, 2, 4, 8
REDUCTIONS = {"mean": 0, "sum": 1, "mean_elements": 2}

_PKG = os.path.dirname(os.path.abspath(__file__))
_HEADER = os.path.join(os.path.dirname(_PKG), "include", "cutbce.h")


def library_path() -> str:
    return os.path.join(_PKG, "libcutbce.so")


class cutbce_problem(ctypes.Structure):
    _fields_ = [
        ("T", ctypes.c_int64), ("V", ctypes.c_int64), ("D", ctypes.c_int64), ("K", ctypes.c_int64),
        ("dtype", ctypes.c_int32), ("reduction", ctypes.c_int32),
        ("H", ctypes.c_void_p), ("E", ctypes.c_void_p), ("targets", ctypes.c_void_p), ("mask", ctypes.c_void_p),
    ]


class cutbce_options(ctypes.Structure):
    _fields_ = [("metrics", ctypes.c_void_p), ("weights", ctypes.c_void_p), ("grad_dtype", ctypes.c_int32),
                ("accumulate", ctypes.c_int32), ("vocab_offset", ctypes.c_int64), ("V_total", ctypes.c_int64)]


class cutbce_grad_options(ctypes.Structure):
    _fields_ = [("grad_dtype", ctypes.c_int32), ("accumulate", ctypes.c_int32)]


class cutbce_distill_problem(ctypes.Structure):
    _fields_ = [
        ("T", ctypes.c_int64), ("V", ctypes.c_int64), ("D", ctypes.c_int64), ("K", ctypes.c_int64),
        ("dtype", ctypes.c_int32), ("reduction", ctypes.c_int32),
        ("H", ctypes.c_void_p), ("E", ctypes.c_void_p), ("ids", ctypes.c_void_p), ("logits", ctypes.c_void_p),
        ("mask", ctypes.c_void_p), ("weights", ctypes.c_void_p), ("temperature", ctypes.c_float),
    ]


class cutbce_preference_problem(ctypes.Structure):
    _fields_ = [
        ("T", ctypes.c_int64), ("V", ctypes.c_int64), ("D", ctypes.c_int64), ("P", ctypes.c_int64),
        ("dtype", ctypes.c_int32), ("reduction", ctypes.c_int32),
        ("H", ctypes.c_void_p), ("E", ctypes.c_void_p), ("ids", ctypes.c_void_p), ("offsets", ctypes.c_void_p),
        ("ref_logp", ctypes.c_void_p), ("mask", ctypes.c_void_p), ("beta", ctypes.c_float),
    ]


GRAD_F32, GRAD_BF16 = 0, 1
ACCUMULATE_DH, ACCUMULATE_DE = 1, 2


def make_options(metrics: Optional[torch.Tensor] = None, weights: Optional[torch.Tensor] = None,
                 grad_dtype: int = GRAD_F32, accumulate: int = 0, vocab_offset: int = 0,
                 V_total: int = 0) -> cutbce_options:
    """Options of cutbce_forward_backward_ex (see include/cutbce.h): metrics is an int32 [T, 4]
    device tensor, weights a float32 [T] device tensor."""
    if metrics is not None and (metrics.dtype != torch.int32 or not metrics.is_contiguous()):
        raise ValueError("metrics must be a contiguous int32 [T, 4] tensor")
    if weights is not None and (weights.dtype != torch.float32 or not weights.is_contiguous()):
        raise ValueError("weights must be a contiguous float32 [T] tensor")
    return cutbce_options(metrics.data_ptr() if metrics is not None else None,
                          weights.data_ptr() if weights is not None else None,
                          int(grad_dtype), int(accumulate), int(vocab_offset), int(V_total))


class CutBCEError(RuntimeError):
    def __init__(self, status: int, where: str = ""):
        self.status = int(status)
        msg = _LIB.cutbce_status_string(self.status).decode() if _LIB is not None else str(status)
        super().__init__(f"{where}: {msg} (status {self.status})" if where else f"{msg} (status {self.status})")


_LIB: Optional[ctypes.CDLL] = None
_P = ctypes.POINTER(cutbce_problem)
_vp, _sz, _i32, _i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64
_SIGS = {
    "cutbce_workspace_size": (_i32, [_P, ctypes.POINTER(_sz)]),
    "cutbce_workspace_size_for": (_i32, [_P, ctypes.c_int, ctypes.POINTER(_sz)]),
    "cutbce_forward": (_i32, [_P, _vp, _sz, _vp, _vp]),
    "cutbce_forward_fixed_scratch": (_i32, [_P, _vp, _vp]),
    "cutbce_backward": (_i32, [_P, _vp, _vp, _vp, _vp, _sz, _vp]),
    "cutbce_forward_backward": (_i32, [_P, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "cutbce_forward_backward_ex": (_i32, [_P, ctypes.POINTER(cutbce_options), _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "cutbce_workspace_size_ex": (_i32, [_P, ctypes.POINTER(cutbce_options), ctypes.c_int, ctypes.POINTER(_sz)]),
    "cutbce_host_buffer_size": (_i32, [_P, ctypes.POINTER(_sz)]),
    "cutbce_forward_backward_host": (_i32, [_P, ctypes.c_float, _vp, _vp, _vp, _vp, _sz, _vp]),
    "cutbce_read_status": (_i32, [_vp, _vp]),
    "cutbce_read_counts": (_i32, [_P, _vp, ctypes.POINTER(_i64), ctypes.POINTER(_i64), _vp, _vp]),
    "cutbce_kernel_launches": (ctypes.c_int, [_P, ctypes.c_int]),
    "cutbce_status_string": (ctypes.c_char_p, [_i32]),
    "cutbce_selftest_wait_timeout": (_i32, [_i64, _vp, _vp]),
    "cutbce_selftest_element_math": (_i32, [_vp, _vp, _i64, _vp]),
    "cutbce_topk_workspace_size": (_i32, [_i64, _i64, _i64, ctypes.c_int, ctypes.POINTER(_sz)]),
    "cutbce_topk": (_i32, [_vp, _i64, _vp, _i64, _i64, _i32, ctypes.c_int, _vp, _vp, _vp, _sz, _vp]),
    "cutbce_hit_at_k": (_i32, [_vp, _i64, ctypes.c_int, _vp, _i64, _vp, _vp]),
    "cutbce_profile_enable": (_i32, [ctypes.c_int]),
    "cutbce_profile_read": (_i32, [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(_i64), ctypes.c_int]),
    "cutbce_probe_scratch_bytes": (_sz, []),
    "cutbce_probe_pipe_rate": (_i32, [ctypes.c_int, _vp, _sz, ctypes.POINTER(ctypes.c_double), _vp]),
    "cutbce_embed_forward": (_i32, [_vp, _i64, _i64, _i32, _vp, _i64, ctypes.c_float, _vp, _vp, _vp]),
    "cutbce_embed_workspace_size": (_i32, [_i64, _i64, _i64, ctypes.POINTER(_sz)]),
    "cutbce_embed_backward": (_i32, [_vp, _i32, _vp, _i64, _i64, _i64, ctypes.c_float, _vp, _i32, _i32, _vp, _sz, _vp]),
    "cutbce_distill_workspace_size": (_i32, [_vp, ctypes.c_int, ctypes.POINTER(_sz)]),
    "cutbce_distill_forward": (_i32, [_vp, _vp, _vp, _vp, _sz, _vp]),
    "cutbce_distill_backward": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "cutbce_distill_forward_backward": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "cutbce_preference_workspace_size": (_i32, [_vp, ctypes.c_int, ctypes.POINTER(_sz)]),
    "cutbce_preference_forward": (_i32, [_vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "cutbce_preference_backward": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "cutbce_preference_forward_backward": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "cutbce_probe_mma": (_i32, [ctypes.c_int, ctypes.c_int, _i64, _vp, _sz, ctypes.POINTER(ctypes.c_double),
                                ctypes.POINTER(ctypes.c_double), _vp]),
}
PROBES = ["ffma", "ffma2", "ex2", "rcp", "tanh", "lg2", "cvt_bf16x2", "fmax", "add2", "iadd", "prmt",
          "ex2_f16x2", "ex2_bf16x2", "tanh_f16x2", "hfma2", "cvt_f16x2", "ffma_sat", "select", "lop", "fmul2"]
KERNEL_KINDS = ["prep_rows", "prep_scan", "prep_gather", "csc_offsets", "item_pass", "position_pass", "finish",
                "pair_sort", "topk", "topk_merge", "col_sums", "embed", "id_sort", "segment_sum", "head_prep",
                "head_lse_pass", "head_row_pass", "head_item_pass", "head_finish"]


def load_library() -> ctypes.CDLL:
    """Load the in-tree libcutbce.so (built by `python -m vocabulary_label_bce_b200.build`)."""
    global _LIB
    if _LIB is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with `python -m vocabulary_label_bce_b200.build`")
        lib = ctypes.CDLL(path)
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = lib
    return _LIB


def declared_functions() -> list[str]:
    """Names of the functions include/cutbce.h declares."""
    text = open(_HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(cutbce_[a-z_]+)\s*\(", text)))


def _check(status: int, where: str) -> None:
    if status != OK:
        raise CutBCEError(status, where)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None:
            torch.cuda.init()
            return _raw_stream(torch._C._cuda_getDevice())
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def make_problem(H: torch.Tensor, E: torch.Tensor, targets: torch.Tensor, mask: Optional[torch.Tensor] = None,
                 reduction: str | int = "mean") -> cutbce_problem:
    """Describe tensors already on the device.  H [T, D], E [V, D] bf16 or fp32, targets int32 [T, K]."""
    if H.dim() != 2 or E.dim() != 2 or targets.dim() != 2:
        raise ValueError("H, E, targets must be 2-D")
    if H.dtype != E.dtype or H.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("H and E must share dtype bf16 or fp32")
    if targets.dtype != torch.int32:
        raise ValueError("targets must be int32")
    for t in (H, E, targets) + ((mask,) if mask is not None else ()):
        if not t.is_contiguous():
            raise ValueError("inputs must be contiguous")
    if mask is not None and mask.dtype not in (torch.uint8, torch.bool):
        raise ValueError("mask must be uint8 or bool")
    red = REDUCTIONS[reduction] if isinstance(reduction, str) else int(reduction)
    return cutbce_problem(H.shape[0], E.shape[0], H.shape[1], targets.shape[1],
                          BF16 if H.dtype == torch.bfloat16 else F32, red,
                          H.data_ptr(), E.data_ptr(), targets.data_ptr(),
                          mask.data_ptr() if mask is not None else None)


# ---------------------------------------------------------------- one function per C entry point
def cutbce_workspace_size(prob: cutbce_problem) -> int:
    n = _sz(0)
    _check(load_library().cutbce_workspace_size(ctypes.byref(prob), ctypes.byref(n)), "cutbce_workspace_size")
    return int(n.value)


def cutbce_workspace_size_for(prob: cutbce_problem, outputs: int) -> int:
    """Workspace bytes for a call computing only `outputs` (a bitwise or of OUT_LOSS, OUT_DH, OUT_DE)."""
    n = _sz(0)
    _check(load_library().cutbce_workspace_size_for(ctypes.byref(prob), int(outputs), ctypes.byref(n)),
           "cutbce_workspace_size_for")
    return int(n.value)


def cutbce_workspace_size_ex(prob: cutbce_problem, opts: Optional[cutbce_options], outputs: int) -> int:
    n = _sz(0)
    _check(load_library().cutbce_workspace_size_ex(ctypes.byref(prob), ctypes.byref(opts) if opts is not None else None,
                                                   int(outputs), ctypes.byref(n)), "cutbce_workspace_size_ex")
    return int(n.value)


def cutbce_forward(prob, ws: torch.Tensor, loss: torch.Tensor, stream=None) -> None:
    _check(load_library().cutbce_forward(ctypes.byref(prob), ws.data_ptr(), ws.numel(), loss.data_ptr(),
                                         _stream(stream)), "cutbce_forward")


# Size of the library's static scratch array (CUTBCE_FIXED_SCRATCH_BYTES in include/cutbce.h).
FIXED_SCRATCH_BYTES = 16 << 20


def cutbce_forward_fixed_scratch(prob, loss: torch.Tensor, stream=None) -> None:
    """Loss only, with the library's static scratch array instead of a workspace (nothing is allocated)."""
    _check(load_library().cutbce_forward_fixed_scratch(ctypes.byref(prob), loss.data_ptr(), _stream(stream)),
           "cutbce_forward_fixed_scratch")


def cutbce_backward(prob, grad_loss: Optional[torch.Tensor], dH: Optional[torch.Tensor],
                    dE: Optional[torch.Tensor], ws: torch.Tensor, stream=None) -> None:
    _check(load_library().cutbce_backward(
        ctypes.byref(prob), grad_loss.data_ptr() if grad_loss is not None else None,
        dH.data_ptr() if dH is not None else None, dE.data_ptr() if dE is not None else None,
        ws.data_ptr(), ws.numel(), _stream(stream)), "cutbce_backward")


def cutbce_forward_backward(prob, grad_loss: Optional[torch.Tensor], loss: Optional[torch.Tensor],
                            dH: Optional[torch.Tensor], dE: Optional[torch.Tensor], ws: torch.Tensor,
                            stream=None) -> None:
    _check(load_library().cutbce_forward_backward(
        ctypes.byref(prob), grad_loss.data_ptr() if grad_loss is not None else None,
        loss.data_ptr() if loss is not None else None, dH.data_ptr() if dH is not None else None,
        dE.data_ptr() if dE is not None else None, ws.data_ptr(), ws.numel(), _stream(stream)),
        "cutbce_forward_backward")


def cutbce_forward_backward_ex(prob, opts: cutbce_options, grad_loss: Optional[torch.Tensor],
                               loss: Optional[torch.Tensor], dH: Optional[torch.Tensor], dE: Optional[torch.Tensor],
                               ws: torch.Tensor, stream=None) -> None:
    _check(load_library().cutbce_forward_backward_ex(
        ctypes.byref(prob), ctypes.byref(opts), grad_loss.data_ptr() if grad_loss is not None else None,
        loss.data_ptr() if loss is not None else None, dH.data_ptr() if dH is not None else None,
        dE.data_ptr() if dE is not None else None, ws.data_ptr(), ws.numel(), _stream(stream)),
        "cutbce_forward_backward_ex")


def cutbce_host_buffer_size(prob: cutbce_problem) -> int:
    n = _sz(0)
    _check(load_library().cutbce_host_buffer_size(ctypes.byref(prob), ctypes.byref(n)), "cutbce_host_buffer_size")
    return int(n.value)


def cutbce_forward_backward_host(prob, grad_loss: float, loss: torch.Tensor, dH: Optional[torch.Tensor],
                                 dE: Optional[torch.Tensor], dev_buf: torch.Tensor, stream=None) -> None:
    """prob's pointers and loss/dH/dE are host (CPU, ideally pinned) tensors; dev_buf is device memory."""
    _check(load_library().cutbce_forward_backward_host(
        ctypes.byref(prob), float(grad_loss), loss.data_ptr(), dH.data_ptr() if dH is not None else None,
        dE.data_ptr() if dE is not None else None, dev_buf.data_ptr(), dev_buf.numel(), _stream(stream)),
        "cutbce_forward_backward_host")


def cutbce_read_status(ws: torch.Tensor, stream=None) -> int:
    return int(load_library().cutbce_read_status(ws.data_ptr(), _stream(stream)))


def cutbce_read_counts(prob, ws: torch.Tensor, row_counts: Optional[torch.Tensor] = None, stream=None):
    nv, npairs = _i64(0), _i64(0)
    _check(load_library().cutbce_read_counts(ctypes.byref(prob), ws.data_ptr(), ctypes.byref(nv),
                                             ctypes.byref(npairs),
                                             row_counts.data_ptr() if row_counts is not None else None,
                                             _stream(stream)), "cutbce_read_counts")
    return int(nv.value), int(npairs.value)


def cutbce_kernel_launches(prob, entry: int) -> int:
    return int(load_library().cutbce_kernel_launches(ctypes.byref(prob), int(entry)))


def cutbce_status_string(status: int) -> str:
    return load_library().cutbce_status_string(int(status)).decode()


def cutbce_selftest_wait_timeout(limit_ns: int, status_dev: torch.Tensor, stream=None) -> None:
    _check(load_library().cutbce_selftest_wait_timeout(int(limit_ns), status_dev.data_ptr(), _stream(stream)),
           "cutbce_selftest_wait_timeout")


def cutbce_selftest_element_math(x: torch.Tensor, stream=None) -> torch.Tensor:
    """[5, n] device tensor: FMA-pipe 2^x, SFU 2^x, FMA-pipe sigmoid(x), sigmoid(x) from
    tanh, and w = 1 + |tanh(x/2)| (see include/cutbce.h)."""
    if x.dtype != torch.float32 or not x.is_contiguous():
        raise ValueError("x must be a contiguous float32 tensor")
    out = torch.empty((5, x.numel()), dtype=torch.float32, device=x.device)
    _check(load_library().cutbce_selftest_element_math(x.data_ptr(), out.data_ptr(), x.numel(), _stream(stream)),
           "cutbce_selftest_element_math")
    return out


def cutbce_topk_workspace_size(B: int, V: int, D: int, k: int) -> int:
    n = _sz(0)
    _check(load_library().cutbce_topk_workspace_size(int(B), int(V), int(D), int(k), ctypes.byref(n)),
           "cutbce_topk_workspace_size")
    return int(n.value)


def cutbce_topk(Q: torch.Tensor, E: torch.Tensor, k: int, ws: Optional[torch.Tensor] = None, stream=None):
    """(ids int32 [B, k], scores float32 [B, k]) of the k best items of every query row of Q (bf16 [B, D])."""
    if Q.dtype != torch.bfloat16 or E.dtype != torch.bfloat16 or not (Q.is_contiguous() and E.is_contiguous()):
        raise ValueError("Q and E must be contiguous bf16 tensors")
    B, D = Q.shape
    V = E.shape[0]
    if ws is None:
        ws = torch.empty(cutbce_topk_workspace_size(B, V, D, k), dtype=torch.uint8, device=Q.device)
    ids = torch.empty((B, k), dtype=torch.int32, device=Q.device)
    scores = torch.empty((B, k), dtype=torch.float32, device=Q.device)
    _check(load_library().cutbce_topk(Q.data_ptr(), B, E.data_ptr(), V, D, BF16, int(k), ids.data_ptr(),
                                      scores.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream)), "cutbce_topk")
    return ids, scores


def cutbce_hit_at_k(ids: torch.Tensor, targets: torch.Tensor, stream=None) -> torch.Tensor:
    """int32 [B]: 1 where one of the query's target ids (-1 = empty) is among its ranked ids."""
    B, k = ids.shape
    hits = torch.empty(B, dtype=torch.int32, device=ids.device)
    _check(load_library().cutbce_hit_at_k(ids.data_ptr(), B, int(k), targets.data_ptr(), targets.shape[1],
                                          hits.data_ptr(), _stream(stream)), "cutbce_hit_at_k")
    return hits


# ---------------------------------------------------------------- item rows
_DTYPES = {torch.bfloat16: BF16, torch.float32: F32}
_GRADS = {torch.float32: GRAD_F32, torch.bfloat16: GRAD_BF16}


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _dense(t: Optional[torch.Tensor], name: str, dtypes, shape=None) -> None:
    """Raises unless t is None or a contiguous tensor of one of `dtypes` (and of `shape`)."""
    if t is None or (t.dtype in dtypes and t.is_contiguous() and (shape is None or t.shape == shape)):
        return
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, not {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")


def _same_device(*tensors: Optional[torch.Tensor]) -> None:
    index = None
    for t in tensors:
        if t is None:
            continue
        if index is None:
            index = t.get_device()
        elif t.get_device() != index:
            raise ValueError(f"all tensors must be on one device, not {[str(x.device) for x in tensors if x is not None]}")


def cutbce_embed_forward(E: torch.Tensor, ids: torch.Tensor, X: torch.Tensor, scale: float = 1.0,
                         status: Optional[torch.Tensor] = None, stream=None) -> None:
    """X[n] = scale * E[ids[n]] (E [V, D] and X ids.shape + [D] bf16 or fp32, ids int32, -1 empty)."""
    i, dtype = E.get_device(), E.dtype
    V, D = E.shape
    n = ids.numel()
    if not (dtype in _DTYPES and ids.dtype is torch.int32 and X.dtype is dtype and E.is_contiguous()
            and ids.is_contiguous() and X.is_contiguous() and X.numel() == n * D and X.shape[-1] == D
            and ids.get_device() == i and X.get_device() == i and status is None):
        _dense(E, "E", tuple(_DTYPES))
        _dense(ids, "ids", (torch.int32,))
        _dense(X, "X", (dtype,), ids.shape + E.shape[1:])
        _dense(status, "status", (torch.int32,))
        _same_device(E, ids, X, status)
    _check((_LIB or load_library()).cutbce_embed_forward(
        E.data_ptr(), V, D, _DTYPES[dtype], ids.data_ptr(), n, float(scale), X.data_ptr(), _ptr(status),
        _stream(stream)), "cutbce_embed_forward")


def cutbce_embed_workspace_size(N: int, V: int, D: int) -> int:
    n = _sz(0)
    _check(load_library().cutbce_embed_workspace_size(int(N), int(V), int(D), ctypes.byref(n)),
           "cutbce_embed_workspace_size")
    return int(n.value)


def cutbce_embed_backward(dX: torch.Tensor, ids: torch.Tensor, dE: torch.Tensor, ws: torch.Tensor, scale: float = 1.0,
                          accumulate: bool = False, stream=None) -> None:
    """dE[v] (+)= scale * sum of dX[n] over ids[n] = v (dX [N, D], dE [V, D] bf16 or fp32)."""
    _dense(dX, "dX", tuple(_DTYPES))
    _dense(ids, "ids", (torch.int32,))
    _dense(dE, "dE", tuple(_GRADS))
    if dX.dim() != 2 or dE.dim() != 2 or dX.shape[0] != ids.numel() or dX.shape[1] != dE.shape[1]:
        raise ValueError("dX [N, D], ids [N] and dE [V, D] do not fit")
    _same_device(dX, ids, dE, ws)
    _check(load_library().cutbce_embed_backward(
        dX.data_ptr(), _DTYPES[dX.dtype], ids.data_ptr(), ids.numel(), dE.shape[0], dE.shape[1], float(scale),
        dE.data_ptr(), _GRADS[dE.dtype], 1 if accumulate else 0, ws.data_ptr(), ws.numel(), _stream(stream)),
        "cutbce_embed_backward")


# ---------------------------------------------------------------- softmax losses
_HEAD_REDUCTIONS = {"mean": 0, "sum": 1}


def _head_ok(H, E, ids, mask, i: int) -> bool:
    """Whether H, E, ids and mask are what the softmax losses take (one pass over the common case)."""
    bf = torch.bfloat16
    return (H.dtype is bf and E.dtype is bf and ids.dtype is torch.int32 and H.dim() == 2 and E.dim() == 2
            and H.shape[1] == E.shape[1] and H.is_contiguous() and E.is_contiguous() and ids.is_contiguous()
            and E.get_device() == i and ids.get_device() == i
            and (mask is None or ((mask.dtype is torch.uint8 or mask.dtype is torch.bool) and mask.is_contiguous()
                                  and mask.shape == H.shape[:1] and mask.get_device() == i)))


def _head_tensors(H, E, ids, mask):
    """Raises for what _head_ok refuses."""
    if H.dim() != 2 or E.dim() != 2 or H.shape[1] != E.shape[1]:
        raise ValueError("H [T, D] and E [V, D] do not fit")
    _dense(H, "H", (torch.bfloat16,))
    _dense(E, "E", (torch.bfloat16,))
    _dense(ids, "ids", (torch.int32,))
    _dense(mask, "mask", (torch.uint8, torch.bool), (H.shape[0],))
    _same_device(H, E, ids, mask)


def _head_reduction(reduction) -> int:
    if reduction not in _HEAD_REDUCTIONS:
        raise ValueError("reduction must be 'mean' or 'sum'")
    return _HEAD_REDUCTIONS[reduction]


def make_distill_problem(H: torch.Tensor, E: torch.Tensor, ids: torch.Tensor, logits: torch.Tensor,
                         mask: Optional[torch.Tensor] = None, weights: Optional[torch.Tensor] = None,
                         temperature: float = 1.0, reduction: str = "mean") -> cutbce_distill_problem:
    """H [T, D], E [V, D] bf16; teacher ids int32 [T, K] and logits float32 [T, K]; mask [T]; weights float32 [T]."""
    i = H.get_device()
    if not _head_ok(H, E, ids, mask, i):
        _head_tensors(H, E, ids, mask)
    if ids.dim() != 2 or ids.shape[0] != H.shape[0]:
        raise ValueError("ids must be [T, K]")
    _dense(logits, "logits", (torch.float32,), ids.shape)
    _dense(weights, "weights", (torch.float32,), H.shape[:1])
    if logits.get_device() != i or (weights is not None and weights.get_device() != i):
        _same_device(H, logits, weights)
    return cutbce_distill_problem(H.shape[0], E.shape[0], H.shape[1], ids.shape[1], BF16, _head_reduction(reduction),
                                  H.data_ptr(), E.data_ptr(), ids.data_ptr(), logits.data_ptr(), _ptr(mask),
                                  _ptr(weights), float(temperature))


def make_preference_problem(H: torch.Tensor, E: torch.Tensor, ids: torch.Tensor, offsets: torch.Tensor,
                            ref_logp: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None,
                            beta: float = 0.1, reduction: str = "mean") -> cutbce_preference_problem:
    """H [T, D], E [V, D] bf16; ids int32 [T]; offsets int32 [2P + 1]; ref_logp float32 [2P]; mask [T]."""
    i = H.get_device()
    if not _head_ok(H, E, ids, mask, i):
        _head_tensors(H, E, ids, mask)
    if ids.numel() != H.shape[0]:
        raise ValueError("ids must be [T]")
    _dense(offsets, "offsets", (torch.int32,))
    if offsets.dim() != 1 or offsets.numel() < 3 or offsets.numel() % 2 == 0:
        raise ValueError("offsets must be [2P + 1] with P >= 1")
    P = (offsets.numel() - 1) // 2
    _dense(ref_logp, "ref_logp", (torch.float32,), (2 * P,))
    if offsets.get_device() != i or (ref_logp is not None and ref_logp.get_device() != i):
        _same_device(H, offsets, ref_logp)
    return cutbce_preference_problem(H.shape[0], E.shape[0], H.shape[1], P, BF16, _head_reduction(reduction),
                                     H.data_ptr(), E.data_ptr(), ids.data_ptr(), offsets.data_ptr(), _ptr(ref_logp),
                                     _ptr(mask), float(beta))


def make_grad_options(dH: Optional[torch.Tensor], dE: Optional[torch.Tensor], accumulate: int = 0) -> cutbce_grad_options:
    """Options for these output tensors (both fp32 or both bf16)."""
    kinds = {t.dtype for t in (dH, dE) if t is not None}
    if len(kinds) != 1 or not kinds <= set(_GRADS):
        raise ValueError("dH and dE must both be float32 or both bfloat16")
    for t in (dH, dE):
        if t is not None and not t.is_contiguous():
            raise ValueError("dH and dE must be contiguous")
    return cutbce_grad_options(_GRADS[kinds.pop()], int(accumulate))


def _head_outputs(prob, loss=None, lse=None, logp=None, dH=None, dE=None) -> None:
    """Raises unless the outputs that are given hold what a call on `prob` writes."""
    for t, dtype, n, name in ((loss, torch.float64, 1, "loss"), (lse, torch.float32, prob.T, "lse"),
                              (logp, torch.float32, 2 * getattr(prob, "P", 0), "logp")):
        if t is not None and (t.dtype is not dtype or t.numel() != n or not t.is_contiguous()):
            raise ValueError(f"{name} must be {n} contiguous {dtype} values")
    if dH is not None and dH.numel() != prob.T * prob.D or dE is not None and dE.numel() != prob.V * prob.D:
        raise ValueError("dH must be [T, D] and dE [V, D]")


def _head_size(fn: str, prob, outputs: int) -> int:
    n = _sz(0)
    _check(getattr(load_library(), fn)(ctypes.byref(prob), int(outputs), ctypes.byref(n)), fn)
    return int(n.value)


def cutbce_distill_workspace_size(prob: cutbce_distill_problem, outputs: int) -> int:
    return _head_size("cutbce_distill_workspace_size", prob, outputs)


def cutbce_preference_workspace_size(prob: cutbce_preference_problem, outputs: int) -> int:
    return _head_size("cutbce_preference_workspace_size", prob, outputs)


def cutbce_distill_forward(prob, loss: Optional[torch.Tensor], lse: Optional[torch.Tensor], ws: torch.Tensor,
                           stream=None) -> None:
    _head_outputs(prob, loss, lse)
    _check(load_library().cutbce_distill_forward(ctypes.byref(prob), _ptr(loss), _ptr(lse), ws.data_ptr(), ws.numel(),
                                                 _stream(stream)), "cutbce_distill_forward")


def cutbce_distill_backward(prob, opts: Optional[cutbce_grad_options], lse: torch.Tensor,
                            grad_loss: Optional[torch.Tensor], dH: Optional[torch.Tensor],
                            dE: Optional[torch.Tensor], ws: torch.Tensor, stream=None) -> None:
    _head_outputs(prob, None, lse, None, dH, dE)
    _check(load_library().cutbce_distill_backward(
        ctypes.byref(prob), ctypes.byref(opts) if opts is not None else None, _ptr(lse), _ptr(grad_loss), _ptr(dH),
        _ptr(dE), ws.data_ptr(), ws.numel(), _stream(stream)), "cutbce_distill_backward")


def cutbce_distill_forward_backward(prob, opts: Optional[cutbce_grad_options], grad_loss: Optional[torch.Tensor],
                                    loss: Optional[torch.Tensor], lse: Optional[torch.Tensor],
                                    dH: Optional[torch.Tensor], dE: Optional[torch.Tensor], ws: torch.Tensor,
                                    stream=None) -> None:
    _head_outputs(prob, loss, lse, None, dH, dE)
    _check(load_library().cutbce_distill_forward_backward(
        ctypes.byref(prob), ctypes.byref(opts) if opts is not None else None, _ptr(grad_loss), _ptr(loss), _ptr(lse),
        _ptr(dH), _ptr(dE), ws.data_ptr(), ws.numel(), _stream(stream)), "cutbce_distill_forward_backward")


def cutbce_preference_forward(prob, loss: Optional[torch.Tensor], logp: Optional[torch.Tensor],
                              lse: Optional[torch.Tensor], ws: torch.Tensor, stream=None) -> None:
    _head_outputs(prob, loss, lse, logp)
    _check(load_library().cutbce_preference_forward(ctypes.byref(prob), _ptr(loss), _ptr(logp), _ptr(lse),
                                                    ws.data_ptr(), ws.numel(), _stream(stream)),
           "cutbce_preference_forward")


def cutbce_preference_backward(prob, opts: Optional[cutbce_grad_options], lse: torch.Tensor,
                               grad_loss: Optional[torch.Tensor], dH: Optional[torch.Tensor],
                               dE: Optional[torch.Tensor], ws: torch.Tensor, stream=None) -> None:
    _head_outputs(prob, None, lse, None, dH, dE)
    _check(load_library().cutbce_preference_backward(
        ctypes.byref(prob), ctypes.byref(opts) if opts is not None else None, _ptr(lse), _ptr(grad_loss), _ptr(dH),
        _ptr(dE), ws.data_ptr(), ws.numel(), _stream(stream)), "cutbce_preference_backward")


def cutbce_preference_forward_backward(prob, opts: Optional[cutbce_grad_options], grad_loss: Optional[torch.Tensor],
                                       loss: Optional[torch.Tensor], logp: Optional[torch.Tensor],
                                       lse: Optional[torch.Tensor], dH: Optional[torch.Tensor],
                                       dE: Optional[torch.Tensor], ws: torch.Tensor, stream=None) -> None:
    _head_outputs(prob, loss, lse, logp, dH, dE)
    _check(load_library().cutbce_preference_forward_backward(
        ctypes.byref(prob), ctypes.byref(opts) if opts is not None else None, _ptr(grad_loss), _ptr(loss), _ptr(logp),
        _ptr(lse), _ptr(dH), _ptr(dE), ws.data_ptr(), ws.numel(), _stream(stream)),
        "cutbce_preference_forward_backward")


def cutbce_profile_enable(enable: bool) -> None:
    _check(load_library().cutbce_profile_enable(1 if enable else 0), "cutbce_profile_enable")


def cutbce_profile_read(reset: bool = True) -> dict:
    """{kernel kind: (total ms, launches)} accumulated since the last reset."""
    n = len(KERNEL_KINDS)
    ms = (ctypes.c_double * n)()
    cnt = (_i64 * n)()
    _check(load_library().cutbce_profile_read(ms, cnt, 1 if reset else 0), "cutbce_profile_read")
    return {k: (float(ms[i]), int(cnt[i])) for i, k in enumerate(KERNEL_KINDS)}


def cutbce_probe_scratch_bytes() -> int:
    return int(load_library().cutbce_probe_scratch_bytes())


def cutbce_probe_pipe_rate(op: str | int, scratch: Optional[torch.Tensor] = None, stream=None) -> float:
    """Operations of one kind an SM retires per clock (median over SMs)."""
    k = PROBES.index(op) if isinstance(op, str) else int(op)
    if scratch is None:
        scratch = torch.empty(cutbce_probe_scratch_bytes(), dtype=torch.uint8, device="cuda")
    r = ctypes.c_double(0.0)
    _check(load_library().cutbce_probe_pipe_rate(k, scratch.data_ptr(), scratch.numel(), ctypes.byref(r),
                                                 _stream(stream)), "cutbce_probe_pipe_rate")
    return float(r.value)


def cutbce_probe_mma(n: int, a_in_tmem: bool, iters: int = 4096, scratch: Optional[torch.Tensor] = None,
                     stream=None, b_mn_major: bool = False, sm_pair: bool = False) -> tuple[float, float]:
    """(issue cycles, total cycles) per 128 x n x 16 bf16 tcgen05.mma (256 x n x 16
    over an SM pair if sm_pair), median over the issuing CTAs."""
    if scratch is None:
        scratch = torch.empty(cutbce_probe_scratch_bytes(), dtype=torch.uint8, device="cuda")
    a, b = ctypes.c_double(0.0), ctypes.c_double(0.0)
    flags = (1 if a_in_tmem else 0) | (2 if b_mn_major else 0) | (4 if sm_pair else 0)
    _check(load_library().cutbce_probe_mma(int(n), flags, int(iters), scratch.data_ptr(),
                                           scratch.numel(), ctypes.byref(a), ctypes.byref(b), _stream(stream)),
           "cutbce_probe_mma")
    return float(a.value), float(b.value)
