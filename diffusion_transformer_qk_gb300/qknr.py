"""Python binding of libqknr.so (ctypes).

Argument marshalling only: tensors are turned into device pointers, row
strides and the current CUDA stream, and every step of the operation runs
in the library's kernels.  The binding has no fallback: if the library is
missing or cannot be loaded, every call raises.

The operation (per-head RMSNorm of Q and K followed by RoPE, V passed
through) is described in ``include/qknr.h``.
"""
from __future__ import annotations

import ctypes
import glob
import math
import os
import threading
from ctypes import c_char, c_float, c_int32, c_int64, c_size_t, c_uint32, c_uint64, c_void_p
from typing import Optional

import torch

from . import build as _build

# enum values of include/qknr.h
BF16, FP16, FP32 = 0, 1, 2
ROPE = {"interleaved": 0, "rotate_half": 1}
COS_LAYOUT = {"shared_row": 0, "per_head_expanded": 1}
STATUS = {
    0: "QKNR_OK", 1: "QKNR_ERR_NULL", 2: "QKNR_ERR_SHAPE", 3: "QKNR_ERR_ALIGN",
    4: "QKNR_ERR_UNSUPPORTED", 5: "QKNR_ERR_CUDA", 6: "QKNR_ERR_TIMEOUT",
    7: "QKNR_ERR_OVERLAP", 8: "QKNR_ERR_ABI", 9: "QKNR_ERR_BOUNDS",
}
STATUS_BY_NAME = {v: k for k, v in STATUS.items()}
OK, ERR_TIMEOUT = 0, 6
FLAG_TEST_STALL = 0x1
FLAG_NO_OVERLAP = 0x2
FLAG_TEST_SHORT_OUT = 0x4
FLAG_NO_PREFETCH = 0x8
ABI_VERSION = 3

EXPORTS = (
    "qknr_args_init", "qknr_forward", "qknr_query", "qknr_status_string",
    "qknr_last_error", "qknr_abi_version", "qknr_sizeof_args", "qknr_sizeof_launch_info",
    "qknr_adaln_args_init", "qknr_adaln_forward", "qknr_adaln_query", "qknr_adaln_sizeof_args",
    "qknr_gn_args_init", "qknr_gn_workspace_bytes", "qknr_gn_silu_forward", "qknr_gn_sizeof_args",
    "qknr_gn_silu_forward_noalloc", "qknr_gn_query",
    "qknr_host_plan_init", "qknr_host_buffer_bytes", "qknr_forward_host", "qknr_sizeof_host_plan",
    "qknr_ln_args_init", "qknr_ln_forward", "qknr_ln_workspace_bytes", "qknr_ln_backward", "qknr_ln_sizeof_args",
    "qknr_grad_args_init", "qknr_grad_workspace_bytes", "qknr_backward", "qknr_sizeof_grad_args",
    "qknr_attn_args_init", "qknr_attn_workspace_bytes", "qknr_attn_backward_workspace_bytes", "qknr_attn_forward",
    "qknr_attn_backward", "qknr_attn_sizeof_args",
    "qknr_rms_args_init", "qknr_rms_forward", "qknr_rms_workspace_bytes", "qknr_rms_backward", "qknr_rms_sizeof_args",
    "qknr_pack_args_init", "qknr_pack_workspace_bytes", "qknr_pack_backward_workspace_bytes", "qknr_pack_forward",
    "qknr_pack_backward", "qknr_pack_sizeof_args",
    "qknr_prefix_args_init", "qknr_prefix_workspace_bytes", "qknr_prefix_forward", "qknr_prefix_sizeof_args",
)
GN_MODE = {"auto": 0, "fused": 1, "two_pass": 2, "cluster": 3}
GN_FLAG_TEST_NO_RECORDS = 0x2
GN_NOALLOC_SCRATCH_BYTES = 1 << 20
HOST_MAX_BUFFERS = 4
LN_UNIT_OFFSET = 0x10
RMS_UNIT_OFFSET = 0x10
RMS_OUT_SAME, RMS_OUT_E4M3 = 0, 1
RMS_BLOCK = 128


class QknrArgs(ctypes.Structure):
    """Mirror of ``qknr_args``."""

    _fields_ = [
        ("abi_version", c_uint32), ("dtype", c_int32),
        ("q", c_void_p), ("k", c_void_p), ("v", c_void_p),
        ("q_out", c_void_p), ("k_out", c_void_p), ("v_out", c_void_p),
        ("q_stride", c_int64), ("k_stride", c_int64), ("v_stride", c_int64),
        ("q_out_stride", c_int64), ("k_out_stride", c_int64), ("v_out_stride", c_int64),
        ("tokens", c_int64),
        ("n_heads_q", c_int32), ("n_heads_k", c_int32), ("n_heads_v", c_int32),
        ("head_dim", c_int32),
        ("gamma_q", c_void_p), ("gamma_k", c_void_p), ("eps", c_float),
        ("cos", c_void_p), ("sin", c_void_p),
        ("cos_dtype", c_int32), ("cos_layout", c_int32), ("cos_rows", c_int64),
        ("rope_style", c_int32),
        ("dev_status", c_void_p),
        ("ctas_per_sm", c_int32), ("stages", c_int32), ("consumer_warps", c_int32),
        ("group_warps", c_int32), ("flags", c_uint32), ("wait_limit_ns", c_uint64),
    ]


class QknrLaunchInfo(ctypes.Structure):
    """Mirror of ``qknr_launch_info``."""

    _fields_ = [
        ("grid", c_int32), ("block", c_int32), ("dyn_smem", c_int32), ("stages", c_int32),
        ("ctas_per_sm", c_int32), ("consumer_warps", c_int32), ("group_warps", c_int32),
        ("stage_bytes", c_int32),
        ("registers", c_int32), ("num_sms", c_int32), ("prefetch_rows", c_int32), ("kernel", c_char * 96),
    ]

    def as_dict(self):
        d = {name: getattr(self, name) for name, _ in self._fields_}
        d["kernel"] = self.kernel.decode()
        return d


class QknrAdaLNArgs(ctypes.Structure):
    """Mirror of ``qknr_adaln_args``."""

    _fields_ = [
        ("abi_version", c_uint32), ("dtype", c_int32),
        ("x", c_void_p), ("out", c_void_p),
        ("x_stride", c_int64), ("out_stride", c_int64),
        ("tokens", c_int64), ("hidden", c_int32), ("rows_per_batch", c_int64),
        ("scale", c_void_p), ("shift", c_void_p), ("mod_dtype", c_int32), ("mod_stride", c_int64),
        ("eps", c_float), ("dev_status", c_void_p),
        ("ctas_per_sm", c_int32), ("stages", c_int32), ("consumer_warps", c_int32), ("group_warps", c_int32),
        ("flags", c_uint32), ("wait_limit_ns", c_uint64),
    ]


class QknrGnArgs(ctypes.Structure):
    """Mirror of ``qknr_gn_args``."""

    _fields_ = [
        ("abi_version", c_uint32), ("dtype", c_int32),
        ("x", c_void_p), ("out", c_void_p),
        ("n", c_int32), ("c", c_int32), ("h", c_int32), ("w", c_int32), ("groups", c_int32),
        ("gamma", c_void_p), ("beta", c_void_p), ("eps", c_float),
        ("workspace", c_void_p), ("workspace_bytes", c_size_t),
        ("piece_elems", c_int32), ("l2_batch_bytes", c_int64),
        ("dev_status", c_void_p), ("mode", c_int32), ("flags", c_uint32), ("wait_limit_ns", c_uint64),
    ]


class QknrHostPlan(ctypes.Structure):
    """Mirror of ``qknr_host_plan``."""

    _fields_ = [
        ("abi_version", c_uint32), ("n_buffers", c_int32), ("chunk_rows", c_int64),
        ("dev_buffers", c_void_p * HOST_MAX_BUFFERS), ("h2d_stream", c_void_p), ("d2h_stream", c_void_p),
        ("events", c_void_p * (3 * HOST_MAX_BUFFERS + 2)),
        ("host_gamma_q", c_void_p), ("host_gamma_k", c_void_p), ("host_cos", c_void_p), ("host_sin", c_void_p),
    ]


class QknrLnArgs(ctypes.Structure):
    """Mirror of ``qknr_ln_args``."""

    _fields_ = [
        ("abi_version", c_uint32), ("dtype", c_int32),
        ("x", c_void_p), ("y", c_void_p),
        ("x_stride", c_int64), ("y_stride", c_int64),
        ("tokens", c_int64), ("hidden", c_int32), ("rows_per_batch", c_int64),
        ("weight", c_void_p), ("bias", c_void_p), ("param_dtype", c_int32), ("param_stride", c_int64),
        ("eps", c_float), ("mean", c_void_p), ("rstd", c_void_p),
        ("dy", c_void_p), ("dx", c_void_p),
        ("dy_stride", c_int64), ("dx_stride", c_int64),
        ("dweight", c_void_p), ("dbias", c_void_p),
        ("workspace", c_void_p), ("workspace_bytes", c_size_t),
        ("dev_status", c_void_p), ("flags", c_uint32), ("wait_limit_ns", c_uint64),
    ]


class QknrGradArgs(ctypes.Structure):
    """Mirror of ``qknr_grad_args``."""

    _fields_ = [
        ("abi_version", c_uint32), ("dtype", c_int32),
        ("q", c_void_p), ("k", c_void_p), ("dq", c_void_p), ("dk", c_void_p), ("dv", c_void_p),
        ("dq_out", c_void_p), ("dk_out", c_void_p), ("dv_out", c_void_p),
        ("q_stride", c_int64), ("k_stride", c_int64),
        ("dq_stride", c_int64), ("dk_stride", c_int64), ("dv_stride", c_int64),
        ("dq_out_stride", c_int64), ("dk_out_stride", c_int64), ("dv_out_stride", c_int64),
        ("tokens", c_int64),
        ("n_heads_q", c_int32), ("n_heads_k", c_int32), ("n_heads_v", c_int32), ("head_dim", c_int32),
        ("gamma_q", c_void_p), ("gamma_k", c_void_p), ("eps", c_float),
        ("cos", c_void_p), ("sin", c_void_p),
        ("cos_dtype", c_int32), ("cos_layout", c_int32), ("cos_rows", c_int64), ("rope_style", c_int32),
        ("dgamma_q", c_void_p), ("dgamma_k", c_void_p),
        ("workspace", c_void_p), ("workspace_bytes", c_size_t),
        ("dev_status", c_void_p), ("flags", c_uint32),
    ]


class QknrAttnArgs(ctypes.Structure):
    """Mirror of ``qknr_attn_args``."""

    _fields_ = [
        ("abi_version", c_uint32), ("dtype", c_int32),
        ("q", c_void_p), ("k", c_void_p), ("v", c_void_p), ("o", c_void_p), ("lse", c_void_p),
        ("q_stride", c_int64), ("k_stride", c_int64), ("v_stride", c_int64), ("o_stride", c_int64),
        ("batch", c_int32), ("seq_q", c_int32), ("seq_k", c_int32),
        ("n_heads_q", c_int32), ("n_heads_k", c_int32), ("head_dim", c_int32),
        ("q_lens", c_void_p), ("k_lens", c_void_p), ("scale", c_float), ("causal", c_int32),
        ("dout", c_void_p), ("dq", c_void_p), ("dk", c_void_p), ("dv", c_void_p),
        ("dout_stride", c_int64), ("dq_stride", c_int64), ("dk_stride", c_int64), ("dv_stride", c_int64),
        ("workspace", c_void_p), ("workspace_bytes", c_size_t),
        ("dev_status", c_void_p), ("flags", c_uint32), ("wait_limit_ns", c_uint64),
    ]


class QknrRmsArgs(ctypes.Structure):
    """Mirror of ``qknr_rms_args``."""

    _fields_ = [
        ("abi_version", c_uint32), ("dtype", c_int32),
        ("x", c_void_p), ("residual", c_void_p), ("sum", c_void_p), ("y", c_void_p),
        ("x_stride", c_int64), ("residual_stride", c_int64), ("sum_stride", c_int64), ("y_stride", c_int64),
        ("tokens", c_int64), ("hidden", c_int32), ("rows_per_batch", c_int64),
        ("weight", c_void_p), ("param_dtype", c_int32), ("param_stride", c_int64),
        ("eps", c_float), ("rstd", c_void_p),
        ("out", c_int32), ("scale_block", c_int32), ("scales", c_void_p),
        ("dy", c_void_p), ("dsum", c_void_p), ("dx", c_void_p),
        ("dy_stride", c_int64), ("dsum_stride", c_int64), ("dx_stride", c_int64),
        ("dweight", c_void_p),
        ("workspace", c_void_p), ("workspace_bytes", c_size_t),
        ("dev_status", c_void_p), ("flags", c_uint32), ("wait_limit_ns", c_uint64),
    ]


class QknrPackArgs(ctypes.Structure):
    """Mirror of ``qknr_pack_args``."""

    _fields_ = [
        ("abi_version", c_uint32), ("dtype", c_int32),
        ("q", c_void_p), ("k", c_void_p), ("v", c_void_p), ("o", c_void_p), ("lse", c_void_p),
        ("q_stride", c_int64), ("k_stride", c_int64), ("v_stride", c_int64), ("o_stride", c_int64),
        ("batch", c_int32), ("rows_q", c_int32), ("rows_k", c_int32),
        ("n_heads_q", c_int32), ("n_heads_k", c_int32), ("head_dim", c_int32),
        ("q_starts", c_void_p), ("k_starts", c_void_p), ("scale", c_float), ("causal", c_int32),
        ("dout", c_void_p), ("dq", c_void_p), ("dk", c_void_p), ("dv", c_void_p),
        ("dout_stride", c_int64), ("dq_stride", c_int64), ("dk_stride", c_int64), ("dv_stride", c_int64),
        ("workspace", c_void_p), ("workspace_bytes", c_size_t),
        ("dev_status", c_void_p), ("flags", c_uint32), ("wait_limit_ns", c_uint64),
    ]


class QknrPrefixArgs(ctypes.Structure):
    """Mirror of ``qknr_prefix_args``."""

    _fields_ = [
        ("abi_version", c_uint32), ("dtype", c_int32),
        ("q", c_void_p), ("k", c_void_p), ("v", c_void_p), ("prefix_k", c_void_p), ("prefix_v", c_void_p),
        ("o", c_void_p), ("lse", c_void_p),
        ("q_stride", c_int64), ("k_stride", c_int64), ("v_stride", c_int64),
        ("prefix_k_stride", c_int64), ("prefix_v_stride", c_int64), ("o_stride", c_int64),
        ("batch", c_int32), ("seq_q", c_int32), ("seq_k", c_int32), ("prefix", c_int32),
        ("n_heads_q", c_int32), ("n_heads_k", c_int32), ("head_dim", c_int32),
        ("q_lens", c_void_p), ("k_lens", c_void_p), ("scale", c_float), ("causal", c_int32),
        ("workspace", c_void_p), ("workspace_bytes", c_size_t),
        ("dev_status", c_void_p), ("flags", c_uint32), ("wait_limit_ns", c_uint64),
    ]


class QknrError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


_lib = None
_lock = threading.Lock()


def library_path(checked: bool = False) -> str:
    return _build.library_path(checked)


def load(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libqknr.so (once).  Raises if it is missing or malformed."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or library_path()
        if not os.path.exists(p):
            raise RuntimeError(
                f"{p} is not built; build it with diffusion_transformer_qk_gb300.build.build_library()")
        lib = ctypes.CDLL(p)
        lib.qknr_args_init.argtypes = [ctypes.POINTER(QknrArgs)]
        lib.qknr_args_init.restype = None
        lib.qknr_forward.argtypes = [ctypes.POINTER(QknrArgs), c_void_p]
        lib.qknr_forward.restype = c_int32
        lib.qknr_query.argtypes = [ctypes.POINTER(QknrArgs), ctypes.POINTER(QknrLaunchInfo)]
        lib.qknr_query.restype = c_int32
        lib.qknr_status_string.argtypes = [c_int32]
        lib.qknr_status_string.restype = ctypes.c_char_p
        lib.qknr_last_error.argtypes = []
        lib.qknr_last_error.restype = ctypes.c_char_p
        lib.qknr_abi_version.argtypes = []
        lib.qknr_abi_version.restype = c_int32
        lib.qknr_sizeof_args.restype = c_size_t
        lib.qknr_sizeof_launch_info.restype = c_size_t
        lib.qknr_adaln_args_init.argtypes = [ctypes.POINTER(QknrAdaLNArgs)]
        lib.qknr_adaln_args_init.restype = None
        lib.qknr_adaln_forward.argtypes = [ctypes.POINTER(QknrAdaLNArgs), c_void_p]
        lib.qknr_adaln_forward.restype = c_int32
        lib.qknr_adaln_query.argtypes = [ctypes.POINTER(QknrAdaLNArgs), ctypes.POINTER(QknrLaunchInfo)]
        lib.qknr_adaln_query.restype = c_int32
        lib.qknr_adaln_sizeof_args.restype = c_size_t
        lib.qknr_gn_args_init.argtypes = [ctypes.POINTER(QknrGnArgs)]
        lib.qknr_gn_args_init.restype = None
        lib.qknr_gn_workspace_bytes.argtypes = [ctypes.POINTER(QknrGnArgs), ctypes.POINTER(c_size_t)]
        lib.qknr_gn_workspace_bytes.restype = c_int32
        lib.qknr_gn_silu_forward.argtypes = [ctypes.POINTER(QknrGnArgs), c_void_p]
        lib.qknr_gn_silu_forward.restype = c_int32
        lib.qknr_gn_sizeof_args.restype = c_size_t
        lib.qknr_gn_silu_forward_noalloc.argtypes = [ctypes.POINTER(QknrGnArgs), c_void_p]
        lib.qknr_gn_silu_forward_noalloc.restype = c_int32
        lib.qknr_gn_query.argtypes = [ctypes.POINTER(QknrGnArgs), ctypes.POINTER(QknrLaunchInfo)]
        lib.qknr_gn_query.restype = c_int32
        lib.qknr_host_plan_init.argtypes = [ctypes.POINTER(QknrHostPlan)]
        lib.qknr_host_plan_init.restype = None
        lib.qknr_host_buffer_bytes.argtypes = [ctypes.POINTER(QknrArgs), ctypes.POINTER(QknrHostPlan),
                                               ctypes.POINTER(c_size_t)]
        lib.qknr_host_buffer_bytes.restype = c_int32
        lib.qknr_forward_host.argtypes = [ctypes.POINTER(QknrArgs), ctypes.POINTER(QknrHostPlan), c_void_p]
        lib.qknr_forward_host.restype = c_int32
        lib.qknr_sizeof_host_plan.restype = c_size_t
        for name, struct in (("ln", QknrLnArgs), ("grad", QknrGradArgs), ("rms", QknrRmsArgs)):
            p_struct = ctypes.POINTER(struct)
            init, space = getattr(lib, f"qknr_{name}_args_init"), getattr(lib, f"qknr_{name}_workspace_bytes")
            init.argtypes, init.restype = [p_struct], None
            space.argtypes, space.restype = [p_struct, ctypes.POINTER(c_size_t)], c_int32
        for fn, struct in ((lib.qknr_ln_forward, QknrLnArgs), (lib.qknr_ln_backward, QknrLnArgs),
                           (lib.qknr_backward, QknrGradArgs), (lib.qknr_rms_forward, QknrRmsArgs),
                           (lib.qknr_rms_backward, QknrRmsArgs)):
            fn.argtypes, fn.restype = [ctypes.POINTER(struct), c_void_p], c_int32
        p_attn = ctypes.POINTER(QknrAttnArgs)
        lib.qknr_attn_args_init.argtypes, lib.qknr_attn_args_init.restype = [p_attn], None
        for fn in (lib.qknr_attn_workspace_bytes, lib.qknr_attn_backward_workspace_bytes):
            fn.argtypes, fn.restype = [p_attn, ctypes.POINTER(c_size_t)], c_int32
        for fn in (lib.qknr_attn_forward, lib.qknr_attn_backward):
            fn.argtypes, fn.restype = [p_attn, c_void_p], c_int32
        lib.qknr_attn_sizeof_args.restype = c_size_t
        lib.qknr_ln_sizeof_args.restype = c_size_t
        lib.qknr_sizeof_grad_args.restype = c_size_t
        lib.qknr_rms_sizeof_args.restype = c_size_t
        for name, struct, fns in (("pack", QknrPackArgs, ("forward", "backward")), ("prefix", QknrPrefixArgs, ("forward",))):
            p_struct = ctypes.POINTER(struct)
            init = getattr(lib, f"qknr_{name}_args_init")
            init.argtypes, init.restype = [p_struct], None
            getattr(lib, f"qknr_{name}_sizeof_args").restype = c_size_t
            for way in fns:
                fn = getattr(lib, f"qknr_{name}_{way}")
                fn.argtypes, fn.restype = [p_struct, c_void_p], c_int32
                space = getattr(lib, f"qknr_{name}_" + ("backward_" if way == "backward" else "") + "workspace_bytes")
                space.argtypes, space.restype = [p_struct, ctypes.POINTER(c_size_t)], c_int32
        if lib.qknr_abi_version() != ABI_VERSION:
            raise RuntimeError("libqknr.so ABI version mismatch")
        if lib.qknr_sizeof_args() != ctypes.sizeof(QknrArgs) or \
                lib.qknr_sizeof_launch_info() != ctypes.sizeof(QknrLaunchInfo) or \
                lib.qknr_adaln_sizeof_args() != ctypes.sizeof(QknrAdaLNArgs) or \
                lib.qknr_gn_sizeof_args() != ctypes.sizeof(QknrGnArgs) or \
                lib.qknr_ln_sizeof_args() != ctypes.sizeof(QknrLnArgs) or \
                lib.qknr_sizeof_grad_args() != ctypes.sizeof(QknrGradArgs) or \
                lib.qknr_attn_sizeof_args() != ctypes.sizeof(QknrAttnArgs) or \
                lib.qknr_rms_sizeof_args() != ctypes.sizeof(QknrRmsArgs) or \
                lib.qknr_pack_sizeof_args() != ctypes.sizeof(QknrPackArgs) or \
                lib.qknr_prefix_sizeof_args() != ctypes.sizeof(QknrPrefixArgs) or \
                lib.qknr_sizeof_host_plan() != ctypes.sizeof(QknrHostPlan):
            raise RuntimeError("libqknr.so struct layout differs from the binding")
        if path is None:
            _lib = lib
        return lib


def last_error() -> str:
    return load().qknr_last_error().decode()


# ---------------------------------------------------------------------------
# marshalling helpers

_ACT = {torch.bfloat16: BF16, torch.float16: FP16}
_TAB = {torch.float32: FP32, torch.bfloat16: BF16}


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _rows(t: Optional[torch.Tensor], name: str) -> int:
    """Row stride (elements) of a 2-D activation view with unit inner stride."""
    if t is None:
        return 0
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D [tokens, heads*head_dim]")
    if t.stride(1) != 1:
        raise ValueError(f"{name} rows must be contiguous")
    if t.stride(0) == 0 and t.shape[0] > 1 and t.numel():
        # to the library 0 is the default stride, and rows that are not there
        raise ValueError(f"{name} is one row expanded to several: pass its contiguous() copy")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.stride(0)


_status_bufs = {}


def status_buffer(device=None) -> torch.Tensor:
    """The per-device int32 status word the binding passes by default."""
    dev = torch.device("cuda", torch.cuda.current_device() if device is None else torch.device(device).index)
    buf = _status_bufs.get(dev.index)
    if buf is None:
        buf = torch.zeros(1, dtype=torch.int32, device=dev)
        _status_bufs[dev.index] = buf
    return buf


def read_status(device=None, reset: bool = True) -> int:
    """Synchronise and return the kernel-side status word (0 = no timeout)."""
    buf = status_buffer(device)
    v = int(buf.item())
    if reset and v:
        buf.zero_()
    return v


def make_args(
    *,
    q: Optional[torch.Tensor] = None,
    k: Optional[torch.Tensor] = None,
    v: Optional[torch.Tensor] = None,
    q_out: Optional[torch.Tensor] = None,
    k_out: Optional[torch.Tensor] = None,
    v_out: Optional[torch.Tensor] = None,
    n_heads_q: int = 0,
    n_heads_k: int = 0,
    n_heads_v: int = 0,
    head_dim: int,
    gamma_q: Optional[torch.Tensor] = None,
    gamma_k: Optional[torch.Tensor] = None,
    cos: Optional[torch.Tensor] = None,
    sin: Optional[torch.Tensor] = None,
    rope_style: str = "interleaved",
    cos_layout: str = "shared_row",
    cos_rows: Optional[int] = None,
    eps: float = 1e-6,
    tokens: Optional[int] = None,
    dev_status: Optional[torch.Tensor] = None,
    ctas_per_sm: int = 0,
    stages: int = 0,
    consumer_warps: int = 0,
    group_warps: int = 0,
    flags: int = 0,
    wait_limit_ns: int = 0,
) -> QknrArgs:
    """Build a ``QknrArgs`` from tensors (no checks beyond marshalling; the
    library validates)."""
    a = QknrArgs()
    load().qknr_args_init(ctypes.byref(a))
    acts = [t for t in (q, k, v) if t is not None]
    if acts:
        dt = acts[0].dtype
        if dt not in _ACT or any(t.dtype != dt for t in acts):
            raise ValueError("q, k, v must share one dtype: bfloat16 or float16")
        a.dtype = _ACT[dt]
    for out, inp, name in ((q_out, q, "q_out"), (k_out, k, "k_out"), (v_out, v, "v_out")):
        if out is not None and inp is not None and out.dtype != inp.dtype:
            raise ValueError(f"{name} dtype differs from its input")
    a.q, a.k, a.v = _ptr(q), _ptr(k), _ptr(v)
    a.q_out, a.k_out, a.v_out = _ptr(q_out), _ptr(k_out), _ptr(v_out)
    a.q_stride, a.k_stride, a.v_stride = _rows(q, "q"), _rows(k, "k"), _rows(v, "v")
    a.q_out_stride = _rows(q_out, "q_out")
    a.k_out_stride = _rows(k_out, "k_out")
    a.v_out_stride = _rows(v_out, "v_out")
    if tokens is None:
        tokens = acts[0].shape[0] if acts else 0
    a.tokens = tokens
    a.n_heads_q, a.n_heads_k, a.n_heads_v, a.head_dim = n_heads_q, n_heads_k, n_heads_v, head_dim
    for g, name in ((gamma_q, "gamma_q"), (gamma_k, "gamma_k")):
        if g is not None and (g.dtype != torch.float32 or not g.is_cuda or not g.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous float32 CUDA tensor")
    a.gamma_q, a.gamma_k = _ptr(gamma_q), _ptr(gamma_k)
    a.eps = eps
    if cos is not None:
        if cos.dtype not in _TAB or sin is None or sin.dtype != cos.dtype:
            raise ValueError("cos and sin must both be float32 or both bfloat16")
        if not (cos.is_contiguous() and sin.is_contiguous() and cos.is_cuda and sin.is_cuda):
            raise ValueError("cos and sin must be contiguous CUDA tensors")
        if cos.shape != sin.shape:
            raise ValueError("cos and sin shapes differ")
        a.cos_dtype = _TAB[cos.dtype]
        if cos_rows is None:
            cos_rows = cos.shape[0]
    a.cos, a.sin = _ptr(cos), _ptr(sin)
    a.cos_layout = COS_LAYOUT[cos_layout]
    a.cos_rows = cos_rows or 0
    a.rope_style = ROPE[rope_style]
    a.dev_status = _ptr(dev_status)
    a.ctas_per_sm, a.stages, a.consumer_warps, a.group_warps = ctas_per_sm, stages, consumer_warps, group_warps
    a.flags, a.wait_limit_ns = flags, wait_limit_ns
    return a


def launch(a: QknrArgs, stream: Optional[torch.cuda.Stream] = None) -> None:
    """qknr_forward on ``stream`` (default: the current stream)."""
    lib = load()
    s = torch.cuda.current_stream() if stream is None else stream
    st = lib.qknr_forward(ctypes.byref(a), c_void_p(s.cuda_stream))
    if st != OK:
        raise QknrError(st, lib.qknr_last_error().decode())


def query(a: QknrArgs) -> dict:
    """qknr_query: the launch qknr_forward would make, as a dict."""
    lib = load()
    info = QknrLaunchInfo()
    st = lib.qknr_query(ctypes.byref(a), ctypes.byref(info))
    if st != OK:
        raise QknrError(st, lib.qknr_last_error().decode())
    return info.as_dict()


# ---------------------------------------------------------------------------
# convenience forms

def _check_table(cos, head_dim, cos_layout, heads):
    if cos_layout == "shared_row":
        if cos.dim() != 2 or cos.shape[1] != head_dim:
            raise ValueError("shared cos/sin must be [rows, head_dim]")
    else:
        if cos.dim() != 3 or cos.shape[1] != heads or cos.shape[2] != head_dim:
            raise ValueError("expanded cos/sin must be [rows, heads, head_dim]")


def packed_args(qkv, n_heads_q, n_heads_k, n_heads_v, head_dim, gamma_q, gamma_k, cos, sin, *,
                out=None, **kw) -> QknrArgs:
    """Arguments for a packed [T, (Hq+Hk+Hv)*D] activation.  ``out=None``
    normalises Q and K in place and leaves V alone; otherwise ``out`` (same
    shape) receives Q, K and a copy of V."""
    D = head_dim
    width = (n_heads_q + n_heads_k + n_heads_v) * D
    if qkv.dim() != 2 or qkv.shape[1] != width:
        raise ValueError(f"qkv must be [tokens, {width}]")
    _check_table(cos, D, kw.get("cos_layout", "shared_row"), n_heads_q)
    q0, k0, v0, v1 = 0, n_heads_q * D, (n_heads_q + n_heads_k) * D, width
    views = dict(q=qkv[:, q0:k0] if n_heads_q else None,
                 k=qkv[:, k0:v0] if n_heads_k else None,
                 v=qkv[:, v0:v1] if n_heads_v else None)
    if out is not None:
        if out.shape != qkv.shape or out.dtype != qkv.dtype:
            raise ValueError("out must match qkv's shape and dtype")
        views.update(q_out=out[:, q0:k0] if n_heads_q else None,
                     k_out=out[:, k0:v0] if n_heads_k else None,
                     v_out=out[:, v0:v1] if n_heads_v else None)
    return make_args(**views, n_heads_q=n_heads_q, n_heads_k=n_heads_k, n_heads_v=n_heads_v,
                     head_dim=D, gamma_q=gamma_q if n_heads_q else None,
                     gamma_k=gamma_k if n_heads_k else None, cos=cos, sin=sin,
                     tokens=qkv.shape[0], **kw)


def qk_norm_rope_packed(qkv, n_heads_q, n_heads_k, n_heads_v, head_dim, gamma_q, gamma_k, cos, sin, *,
                        out=None, stream=None, status=True, **kw):
    """Fused QK-RMSNorm + RoPE on a packed QKV activation; returns the
    tensor holding the result (``qkv`` itself when in place)."""
    if status and "dev_status" not in kw:
        kw["dev_status"] = status_buffer(qkv.device)
    launch(packed_args(qkv, n_heads_q, n_heads_k, n_heads_v, head_dim, gamma_q, gamma_k, cos, sin,
                       out=out, **kw), stream)
    return qkv if out is None else out


def qk_norm_rope_tensor(x, n_heads, head_dim, gamma, cos, sin, *, out=None, stream=None, status=True,
                        **kw):
    """Per-tensor launch (one separate Q or K tensor [T, H*D]), the form
    of page 2's FLUX.2 integration.  In place unless ``out`` is given."""
    if x.dim() != 2 or x.shape[1] != n_heads * head_dim:
        raise ValueError("x must be [tokens, n_heads*head_dim]")
    _check_table(cos, head_dim, kw.get("cos_layout", "shared_row"), n_heads)
    if status and "dev_status" not in kw:
        kw["dev_status"] = status_buffer(x.device)
    launch(make_args(q=x, q_out=out, n_heads_q=n_heads, head_dim=head_dim, gamma_q=gamma, cos=cos, sin=sin,
                     **kw), stream)
    return x if out is None else out


def qk_norm_rope_separate(q, k, n_heads, head_dim, gamma_q, gamma_k, cos, sin, *, v=None, q_out=None,
                          k_out=None, v_out=None, n_heads_v=None, stream=None, status=True, **kw):
    """Q and K as separate [T, H*D] tensors in one launch (and V copied into
    ``v_out`` when both are given)."""
    _check_table(cos, head_dim, kw.get("cos_layout", "shared_row"), n_heads)
    if status and "dev_status" not in kw:
        kw["dev_status"] = status_buffer(q.device)
    hv = (n_heads if n_heads_v is None else n_heads_v) if (v is not None and v_out is not None) else 0
    launch(make_args(q=q, k=k, v=v if hv else None, q_out=q_out, k_out=k_out, v_out=v_out if hv else None,
                     n_heads_q=n_heads, n_heads_k=n_heads, n_heads_v=hv, head_dim=head_dim,
                     gamma_q=gamma_q, gamma_k=gamma_k, cos=cos, sin=sin, **kw), stream)


# ---------------------------------------------------------------------------
# host-resident activations: qknr_forward_host (include/qknr.h)

_cudart = None


def _cudart_lib() -> ctypes.CDLL:
    """The CUDA runtime libqknr.so links (already loaded with it), for the
    events the host pipeline hands the library."""
    global _cudart
    if _cudart is None:
        load()
        cands = sorted(glob.glob(os.path.join(_build.cuda_lib_dir(), "libcudart.so*")))
        if not cands:
            raise RuntimeError("libcudart.so not found next to the CUDA toolkit")
        lib = ctypes.CDLL(cands[-1])
        lib.cudaEventCreateWithFlags.argtypes = [ctypes.POINTER(c_void_p), c_uint32]
        lib.cudaEventCreateWithFlags.restype = c_int32
        lib.cudaEventDestroy.argtypes = [c_void_p]
        lib.cudaEventDestroy.restype = c_int32
        _cudart = lib
    return _cudart


def host_args(*, q=None, k=None, v=None, q_out=None, k_out=None, v_out=None, n_heads_q=0, n_heads_k=0,
              n_heads_v=0, head_dim, tokens, gamma_q=None, gamma_k=None, cos=None, sin=None, cos_rows=0,
              rope_style="interleaved", cos_layout="shared_row", eps=1e-6, dtype=torch.bfloat16, cos_dtype=FP32,
              dev_status=None, ctas_per_sm=0, stages=0, consumer_warps=0, group_warps=0, flags=0,
              wait_limit_ns=0) -> QknrArgs:
    """``qknr_args`` for qknr_forward_host: q, k, v and the outputs are host
    tensor views ([T, heads*D] rows with unit inner stride) or None; gamma,
    cos and sin are device tensors."""
    a = QknrArgs()
    load().qknr_args_init(ctypes.byref(a))
    a.dtype = _ACT[dtype]
    for name, t in (("q", q), ("k", k), ("v", v), ("q_out", q_out), ("k_out", k_out), ("v_out", v_out)):
        if t is None:
            continue
        if t.is_cuda or t.dim() != 2 or t.stride(1) != 1 or t.dtype != dtype:
            raise ValueError(f"{name} must be a 2-D host tensor of {dtype} with contiguous rows")
        setattr(a, name, t.data_ptr())
        setattr(a, name + "_stride", t.stride(0))
    a.tokens = tokens
    a.n_heads_q, a.n_heads_k, a.n_heads_v, a.head_dim = n_heads_q, n_heads_k, n_heads_v, head_dim
    a.gamma_q, a.gamma_k = _ptr(gamma_q), _ptr(gamma_k)
    a.eps = eps
    a.cos, a.sin = _ptr(cos), _ptr(sin)
    a.cos_dtype = cos_dtype
    a.cos_layout = COS_LAYOUT[cos_layout]
    a.cos_rows = cos_rows
    a.rope_style = ROPE[rope_style]
    a.dev_status = _ptr(dev_status)
    a.ctas_per_sm, a.stages, a.consumer_warps, a.group_warps = ctas_per_sm, stages, consumer_warps, group_warps
    a.flags, a.wait_limit_ns = flags, wait_limit_ns
    return a


class HostPipeline:
    """The fused QK-RMSNorm + RoPE on a packed QKV activation that lives in
    (pinned) host memory, through qknr_forward_host: token rows go through
    device staging buffers in chunks, with the host-to-device copy of one
    chunk, the kernel on the previous one and the device-to-host copy of the
    one before that on three streams.  All of that runs inside the library;
    this class only owns what the library does not allocate (the staging
    buffers and the device copies of the gains and tables, made by torch;
    two copy streams; the events) and marshals the call.

    In place on the host (``out_host`` None or the input) only the Q and K
    columns of each row cross the host link: V is neither read nor written
    by the operation, so it stays where it is.  With a separate ``out_host``
    the Q, K and V columns go both ways and V is copied through unchanged.
    The gains and tables are copied from the host to the device every call.
    Results are bitwise those of ``qk_norm_rope_packed`` on the whole
    activation.
    """

    def __init__(self, width: int, dtype: torch.dtype, chunk_rows: int = 2048, n_buffers: int = 3,
                 device=None):
        lib = load()
        self.device = torch.device("cuda", torch.cuda.current_device() if device is None
                                   else torch.device(device).index)
        if not 1 <= n_buffers <= 4:
            raise ValueError("n_buffers must be 1..4")
        self.chunk_rows = int(chunk_rows)
        self.width = int(width)
        self.dtype = dtype
        self.bufs = [torch.empty(self.chunk_rows * self.width, dtype=dtype, device=self.device)
                     for _ in range(n_buffers)]
        self.h2d = torch.cuda.Stream(self.device)
        self.d2h = torch.cuda.Stream(self.device)
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self.tables = {}
        rt = _cudart_lib()
        self.events = []
        with torch.cuda.device(self.device):
            for _ in range(3 * n_buffers + 2):
                e = c_void_p()
                err = rt.cudaEventCreateWithFlags(ctypes.byref(e), 2)   # cudaEventDisableTiming
                if err != 0:
                    raise RuntimeError(f"cudaEventCreateWithFlags failed with error {err}")
                self.events.append(e.value)
        self.plan = QknrHostPlan()
        lib.qknr_host_plan_init(ctypes.byref(self.plan))
        self.plan.n_buffers = n_buffers
        self.plan.chunk_rows = self.chunk_rows
        for i, b in enumerate(self.bufs):
            self.plan.dev_buffers[i] = b.data_ptr()
        self.plan.h2d_stream = self.h2d.cuda_stream
        self.plan.d2h_stream = self.d2h.cuda_stream
        for i, e in enumerate(self.events):
            self.plan.events[i] = e
        self.last_h2d_bytes = self.last_d2h_bytes = 0

    def __del__(self):
        rt = _cudart
        if rt is not None:
            for e in getattr(self, "events", []):
                rt.cudaEventDestroy(c_void_p(e))

    def _device_table(self, name, t):
        """The device buffer the host table ``t`` is copied into (kept across calls)."""
        d = self.tables.get(name)
        if d is None or d.shape != t.shape or d.dtype != t.dtype:
            d = torch.empty(t.shape, dtype=t.dtype, device=self.device)
            self.tables[name] = d
        return d

    def read_status(self) -> int:
        """Synchronise and return (then clear) the kernels' status word."""
        v = int(self.status.item())
        if v:
            self.status.zero_()
        return v

    def __call__(self, qkv_host, n_heads_q, n_heads_k, n_heads_v, head_dim, gamma_q, gamma_k, cos, sin, *,
                 out_host=None, rope_style="interleaved", cos_layout="shared_row", eps=1e-6, **tune):
        if qkv_host.is_cuda or qkv_host.dim() != 2 or qkv_host.shape[1] != self.width or qkv_host.stride(1) != 1:
            raise ValueError("qkv_host must be a 2-D host tensor of the pipeline's width with contiguous rows")
        if qkv_host.dtype != self.dtype:
            raise ValueError("qkv_host dtype differs from the pipeline's")
        if (n_heads_q + n_heads_k + n_heads_v) * head_dim != self.width:
            raise ValueError("head counts do not match the pipeline's width")
        in_place = out_host is None or out_host.data_ptr() == qkv_host.data_ptr()
        if out_host is not None and (out_host.shape != qkv_host.shape or out_host.dtype != qkv_host.dtype or
                                     out_host.stride(1) != 1):
            raise ValueError("out_host must match qkv_host")
        T, D = qkv_host.shape[0], head_dim
        q0, k0, v0 = 0, n_heads_q * D, (n_heads_q + n_heads_k) * D

        def cols(t, a, b):
            return None if t is None or a == b else t[:, a:b]

        dev = {n: self._device_table(n, t) for n, t in (("gamma_q", gamma_q), ("gamma_k", gamma_k), ("cos", cos),
                                                       ("sin", sin))}
        cos_dtype = _TAB[cos.dtype]
        a = host_args(q=cols(qkv_host, q0, k0), k=cols(qkv_host, k0, v0), v=cols(qkv_host, v0, self.width),
                      q_out=None if in_place else cols(out_host, q0, k0),
                      k_out=None if in_place else cols(out_host, k0, v0),
                      v_out=None if in_place else cols(out_host, v0, self.width),
                      n_heads_q=n_heads_q, n_heads_k=n_heads_k, n_heads_v=n_heads_v, head_dim=D, tokens=T,
                      gamma_q=dev["gamma_q"], gamma_k=dev["gamma_k"], cos=dev["cos"], sin=dev["sin"],
                      cos_rows=cos.shape[0], rope_style=rope_style, cos_layout=cos_layout, eps=eps,
                      dtype=qkv_host.dtype, cos_dtype=cos_dtype, dev_status=self.status, **tune)
        self.plan.host_gamma_q, self.plan.host_gamma_k = gamma_q.data_ptr(), gamma_k.data_ptr()
        self.plan.host_cos, self.plan.host_sin = cos.data_ptr(), sin.data_ptr()
        lib = load()
        stream = torch.cuda.current_stream(self.device)
        st = lib.qknr_forward_host(ctypes.byref(a), ctypes.byref(self.plan), c_void_p(stream.cuda_stream))
        if st != OK:
            raise QknrError(st, lib.qknr_last_error().decode())
        # the host tables and device buffers are in use until the stream's
        # work is done
        for t in list(dev.values()) + self.bufs:
            t.record_stream(stream)
        es = qkv_host.element_size()
        moved = (n_heads_q + n_heads_k + (0 if in_place else n_heads_v)) * D * es * T
        tables = sum(t.numel() * t.element_size() for t in (gamma_q, gamma_k, cos, sin))
        self.last_h2d_bytes = moved + tables
        self.last_d2h_bytes = moved
        return qkv_host if in_place else out_host


# ---------------------------------------------------------------------------
# AdaLN scale/shift (include/qknr_adaln.h)

def adaln_args(x, scale, shift, *, rows_per_batch=None, out=None, eps=1e-6, dev_status=None, ctas_per_sm=0,
               stages=0, consumer_warps=0, group_warps=0, flags=0, wait_limit_ns=0) -> QknrAdaLNArgs:
    """Arguments for ``out = LN(x) * (1 + scale[b]) + shift[b]`` over token
    rows ``x`` [T, C]; ``scale``/``shift`` are [B, C] (fp32 or x's dtype);
    row t belongs to sample t // rows_per_batch (default: one sample)."""
    a = QknrAdaLNArgs()
    load().qknr_adaln_args_init(ctypes.byref(a))
    if x.dtype not in _ACT:
        raise ValueError("x must be bfloat16 or float16")
    a.dtype = _ACT[x.dtype]
    a.x, a.x_stride = x.data_ptr(), _rows(x, "x")
    if out is not None:
        if out.dtype != x.dtype or out.shape != x.shape:
            raise ValueError("out must match x's shape and dtype")
        a.out, a.out_stride = out.data_ptr(), _rows(out, "out")
    a.tokens, a.hidden = x.shape[0], x.shape[1]
    a.rows_per_batch = rows_per_batch or 0
    for m, name in ((scale, "scale"), (shift, "shift")):
        if m.dim() != 2 or m.shape[1] != x.shape[1] or m.dtype != scale.dtype:
            raise ValueError(f"{name} must be [B, C] like scale")
    if scale.dtype == torch.float32:
        a.mod_dtype = FP32
    elif scale.dtype == x.dtype:
        a.mod_dtype = a.dtype
    else:
        raise ValueError("scale/shift must be float32 or x's dtype")
    a.scale, a.shift = scale.data_ptr(), shift.data_ptr()
    if _rows(scale, "scale") != _rows(shift, "shift"):
        raise ValueError("scale and shift need the same row stride")
    a.mod_stride = _rows(scale, "scale")
    a.eps = eps
    a.dev_status = _ptr(dev_status)
    a.ctas_per_sm, a.stages, a.consumer_warps, a.group_warps = ctas_per_sm, stages, consumer_warps, group_warps
    a.flags, a.wait_limit_ns = flags, wait_limit_ns
    return a


def adaln_launch(a: QknrAdaLNArgs, stream: Optional[torch.cuda.Stream] = None) -> None:
    lib = load()
    s = torch.cuda.current_stream() if stream is None else stream
    st = lib.qknr_adaln_forward(ctypes.byref(a), c_void_p(s.cuda_stream))
    if st != OK:
        raise QknrError(st, lib.qknr_last_error().decode())


def adaln_query(a: QknrAdaLNArgs) -> dict:
    lib = load()
    info = QknrLaunchInfo()
    st = lib.qknr_adaln_query(ctypes.byref(a), ctypes.byref(info))
    if st != OK:
        raise QknrError(st, lib.qknr_last_error().decode())
    return info.as_dict()


def adaln_modulate(x, scale, shift, *, rows_per_batch=None, out=None, stream=None, status=True, **kw):
    """AdaLN scale/shift on token rows ``x``; in place unless ``out`` is given."""
    if status and "dev_status" not in kw:
        kw["dev_status"] = status_buffer(x.device)
    adaln_launch(adaln_args(x, scale, shift, rows_per_batch=rows_per_batch, out=out, **kw), stream)
    return x if out is None else out


# ---------------------------------------------------------------------------
# group norm + SiLU (include/qknr_gn.h)

def gn_args(x, groups, gamma, beta, *, out=None, eps=1e-6, workspace=None, piece_elems=0,
            l2_batch_bytes=0, mode="auto", dev_status=None, flags=0, wait_limit_ns=0) -> QknrGnArgs:
    """Arguments for ``silu(group_norm(x))`` on an NCHW tensor ``x``."""
    if x.dim() != 4 or not x.is_contiguous() or not x.is_cuda or x.dtype not in _ACT:
        raise ValueError("x must be a contiguous 4-D (NCHW) bfloat16/float16 CUDA tensor")
    a = QknrGnArgs()
    load().qknr_gn_args_init(ctypes.byref(a))
    a.dtype = _ACT[x.dtype]
    a.x = x.data_ptr()
    if out is not None:
        if out.shape != x.shape or out.dtype != x.dtype or not out.is_contiguous():
            raise ValueError("out must be contiguous and match x")
        a.out = out.data_ptr()
    a.n, a.c, a.h, a.w = x.shape
    a.groups = groups
    for t, name in ((gamma, "gamma"), (beta, "beta")):
        if t.dtype != torch.float32 or not t.is_cuda or t.numel() != x.shape[1] or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous float32 CUDA tensor of C values")
    a.gamma, a.beta = gamma.data_ptr(), beta.data_ptr()
    a.eps = eps
    a.piece_elems, a.l2_batch_bytes = piece_elems, l2_batch_bytes
    a.mode = GN_MODE[mode]
    a.dev_status = _ptr(dev_status)
    a.flags, a.wait_limit_ns = flags, wait_limit_ns
    if workspace is not None:
        a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    return a


def gn_query(a: QknrGnArgs) -> dict:
    """qknr_gn_query: the path and launch qknr_gn_silu_forward would take."""
    lib = load()
    info = QknrLaunchInfo()
    st = lib.qknr_gn_query(ctypes.byref(a), ctypes.byref(info))
    if st != OK:
        raise QknrError(st, lib.qknr_last_error().decode())
    return info.as_dict()


def gn_workspace_bytes(a: QknrGnArgs) -> int:
    lib = load()
    n = c_size_t(0)
    st = lib.qknr_gn_workspace_bytes(ctypes.byref(a), ctypes.byref(n))
    if st != OK:
        raise QknrError(st, lib.qknr_last_error().decode())
    return n.value


def gn_launch(a: QknrGnArgs, stream: Optional[torch.cuda.Stream] = None) -> None:
    lib = load()
    s = torch.cuda.current_stream() if stream is None else stream
    st = lib.qknr_gn_silu_forward(ctypes.byref(a), c_void_p(s.cuda_stream))
    if st != OK:
        raise QknrError(st, lib.qknr_last_error().decode())


def group_norm_silu(x, groups, gamma, beta, *, out=None, workspace=None, stream=None, status=True, **kw):
    """silu(group_norm(x)) on NCHW ``x``; in place unless ``out`` is given.
    ``workspace`` (a CUDA tensor of at least gn_workspace_bytes) is created
    by this binding when not given."""
    if status and "dev_status" not in kw:
        kw["dev_status"] = status_buffer(x.device)
    a = gn_args(x, groups, gamma, beta, out=out, **kw)
    if workspace is None:
        workspace = torch.empty(gn_workspace_bytes(a), dtype=torch.uint8, device=x.device)
    a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    gn_launch(a, stream)
    return x if out is None else out


def gn_launch_noalloc(a: QknrGnArgs, stream: Optional[torch.cuda.Stream] = None) -> None:
    """qknr_gn_silu_forward_noalloc: the group-norm + SiLU call for callers
    that cannot allocate device memory; its statistics scratch is a fixed
    array inside the library (GN_NOALLOC_SCRATCH_BYTES), shared by every
    call on the device, and a.workspace is ignored."""
    lib = load()
    s = torch.cuda.current_stream() if stream is None else stream
    st = lib.qknr_gn_silu_forward_noalloc(ctypes.byref(a), c_void_p(s.cuda_stream))
    if st != OK:
        raise QknrError(st, lib.qknr_last_error().decode())


# ---------------------------------------------------------------------------
# training: helpers of the entry points below
#
# A training step makes the same few calls over and over, so what a call's
# metadata decides (every check of shapes, strides and dtypes, the filled-in
# argument struct, the workspace's size) is worked out once per combination
# and kept; a call then copies the struct and puts its pointers in.  Nothing
# is kept of the tensors themselves.

_byref = ctypes.byref
_plans = {}
_MOST_PLANS = 1024
_FIXED = (int, float, bool, str, tuple, type(None))


class _Plan:
    __slots__ = ("struct", "args", "workspace", "info")

    def __init__(self, a, workspace_fn=None, info=None):
        n = c_size_t(0)
        if workspace_fn is not None:
            st = workspace_fn(ctypes.byref(a), ctypes.byref(n))
            if st != OK:
                raise QknrError(st, load().qknr_last_error().decode())
        self.workspace = n.value
        for name, kind in a._fields_:
            if kind is c_void_p:
                setattr(a, name, None)
        self.struct, self.args, self.info = type(a), bytes(a), info

    def new(self):
        return self.struct.from_buffer_copy(self.args)


def _keep(key, plan):
    if not all(isinstance(x, _FIXED) for x in key):   # a tensor, say: the same object may hold another number
        return plan
    if len(_plans) >= _MOST_PLANS:
        _plans.clear()
    _plans[key] = plan
    return plan


def _meta(t):
    """What a plan depends on of a tensor."""
    return None if t is None else (t.shape, t.stride(), t.dtype, t.get_device())


def _empty(shape, dtype, like, stream):
    """A new tensor on like's device that belongs to the stream the call runs
    on, so that its memory is not handed out again while that stream uses it."""
    if stream is None:
        if dtype is like.dtype and shape == like.shape and like.is_contiguous():
            return torch.empty_like(like)         # half a microsecond less
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _one_device(like, *tensors) -> None:
    device = like.get_device()
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError("all tensors of a call must be on one device")


def _call(fn, a, stream, like) -> None:
    """One library call on ``stream`` (default: the current stream of like's
    device)."""
    device = like.get_device()
    if stream is None:
        s = torch._C._cuda_getCurrentRawStream(device)
    elif stream.device_index == device:
        s = stream.cuda_stream
    else:
        raise ValueError("the stream must be on the tensors' device")
    if torch._C._cuda_getDevice() == device:      # the library launches on the calling thread's device
        st = fn(_byref(a), s)
    else:
        with torch.cuda.device(device):
            st = fn(_byref(a), s)
    if st != OK:
        raise QknrError(st, load().qknr_last_error().decode())


def _workspace(a, plan, workspace, like, stream):
    """Put a workspace into ``a``: the caller's, or a new one.  Returns the
    tensor (to be kept until the call)."""
    if workspace is None:
        if not plan.workspace:
            return None
        workspace = _empty((plan.workspace,), torch.uint8, like, stream)
        a.workspace, a.workspace_bytes = workspace.data_ptr(), plan.workspace
    else:
        if not workspace.is_cuda or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor")
        _one_device(like, workspace)
        a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    return workspace


def _status(a, status, dev_status, like):
    """The status word: the caller's, the device's, or none."""
    if dev_status is not None:
        if dev_status.dtype != torch.int32 or not dev_status.is_cuda or not dev_status.numel():
            raise ValueError("dev_status must be an int32 CUDA tensor")
        _one_device(like, dev_status)
        a.dev_status = dev_status.data_ptr()
    elif status:
        word = _status_bufs.get(like.get_device())
        a.dev_status = (status_buffer(like.device) if word is None else word).data_ptr()


def _stride(t, name):
    """Row stride of a 2-D view; 0 (the library's default) where it means
    nothing: without elements, or with a single row and a stride that would
    not do for several."""
    stride = _rows(t, name) if t.numel() else 0
    return 0 if t.shape[0] == 1 and (stride < t.shape[1] or stride % 8) else stride


def _match(t, like, name):
    if t.dtype != like.dtype or t.shape != like.shape:
        raise ValueError(f"{name} must match {like.dtype} {tuple(like.shape)}")
    return t


def _vector(t, n, name, like=None):
    """A contiguous float32 CUDA tensor of n values (on like's device)."""
    if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous() or t.numel() != n:
        raise ValueError(f"{name} must be a contiguous float32 CUDA tensor of {n} values")
    if like is not None:
        _one_device(like, t)
    return t


# ---------------------------------------------------------------------------
# layer norm and its backward pass (include/qknr_ln.h)

def ln_args(x, weight=None, bias=None, *, rows_per_batch=None, unit_offset=False, eps=1e-6, dev_status=None,
            flags=0, wait_limit_ns=0) -> QknrLnArgs:
    """The arguments both passes share: token rows ``x`` [T, C], ``weight``
    and ``bias`` [C] or [B, C] (float32 or x's dtype; either may be None) and
    which of their rows a token takes (t // rows_per_batch; default: one
    row)."""
    a = QknrLnArgs()
    load().qknr_ln_args_init(ctypes.byref(a))
    if x.dtype not in _ACT:
        raise ValueError("x must be bfloat16 or float16")
    a.dtype = _ACT[x.dtype]
    a.x, a.x_stride = x.data_ptr(), _stride(x, "x")
    a.tokens, a.hidden = x.shape
    a.rows_per_batch = rows_per_batch or 0
    sets = -(-x.shape[0] // rows_per_batch) if rows_per_batch else 1
    for name, t in (("weight", weight), ("bias", bias)):
        if t is None:
            continue
        rows = t.view(1, -1) if t.dim() == 1 else t
        if rows.dim() != 2 or rows.shape[1] != x.shape[1] or rows.shape[0] < sets:
            raise ValueError(f"{name} must be [C] or [{sets}, C]")
        if t.dtype not in (torch.float32, x.dtype) or (weight is not None and t.dtype != weight.dtype):
            raise ValueError("weight and bias must both be float32 or both of x's dtype")
        stride = _stride(rows, name)
        if rows.shape[0] > 1 and a.param_stride and stride != a.param_stride:
            raise ValueError("weight and bias need the same row stride")
        if rows.shape[0] > 1:
            a.param_stride = stride
        a.param_dtype = FP32 if t.dtype == torch.float32 else a.dtype
        setattr(a, name, t.data_ptr())
    a.eps = eps
    a.dev_status = _ptr(dev_status)
    a.flags, a.wait_limit_ns = flags | (LN_UNIT_OFFSET if unit_offset else 0), wait_limit_ns
    return a


def layer_norm(x, weight=None, bias=None, *, rows_per_batch=None, unit_offset=False, out=None, mean=None, rstd=None,
               eps=1e-6, stream=None, status=True, dev_status=None, flags=0, wait_limit_ns=0):
    """Layer norm of token rows ``x`` [T, C] for training: returns (y, mean,
    rstd), the last two float32 [T] for the backward pass.

    ``weight``/``bias`` are [C], or [B, C] with row t taking row
    t // rows_per_batch; with ``unit_offset`` the gain is 1 + weight (the
    modulated norm of ``adaln_modulate``).  The result goes to ``out``, a new
    tensor by default (the backward pass needs x); ``out=x`` is in place."""
    key = ("ln", _meta(x), _meta(weight), _meta(bias), _meta(out), rows_per_batch, unit_offset, eps, flags, wait_limit_ns)
    plan = _plans.get(key)
    if plan is None:
        _one_device(x, weight, bias, out)
        a = ln_args(x, weight, bias, rows_per_batch=rows_per_batch, unit_offset=unit_offset, eps=eps, flags=flags,
                    wait_limit_ns=wait_limit_ns)
        a.y_stride = x.shape[1] if out is None else _stride(_match(out, x, "out"), "out")
        plan = _keep(key, _Plan(a))
    T = x.shape[0]
    if out is None:
        out = _empty(x.shape, x.dtype, x, stream)
    mean = _empty((T,), torch.float32, x, stream) if mean is None else _vector(mean, T, "mean", x)
    rstd = _empty((T,), torch.float32, x, stream) if rstd is None else _vector(rstd, T, "rstd", x)
    a = plan.new()
    a.x, a.y, a.mean, a.rstd = x.data_ptr(), out.data_ptr(), mean.data_ptr(), rstd.data_ptr()
    if weight is not None:
        a.weight = weight.data_ptr()
    if bias is not None:
        a.bias = bias.data_ptr()
    _status(a, status, dev_status, x)
    _call((_lib or load()).qknr_ln_forward, a, stream, x)
    return out, mean, rstd


def layer_norm_backward(dy, x, weight, mean, rstd, *, rows_per_batch=None, unit_offset=False, out=None, dweight=None,
                        dbias=None, workspace=None, stream=None, status=True, dev_status=None, flags=0,
                        wait_limit_ns=0):
    """Gradients of ``layer_norm``: returns (dx, dweight, dbias), the last two
    float32: [C], or a row for each sample where ``rows_per_batch`` is given or
    weight has rows (for its first rows, if x has fewer samples).  ``out``
    receives dx (default: a new tensor; ``out=dy`` is in place)."""
    T, C = x.shape
    if T == 0 and weight is not None and weight.dim() == 1:
        rows_per_batch = None                     # no samples, but a gradient of the one row: zero
    key = ("ln_bwd", _meta(dy), _meta(x), _meta(weight), _meta(out), rows_per_batch, unit_offset, flags,
           wait_limit_ns)
    plan = _plans.get(key)
    if plan is None:
        _one_device(x, dy, weight, out)
        a = ln_args(x, weight, None, rows_per_batch=rows_per_batch, unit_offset=unit_offset, flags=flags,
                    wait_limit_ns=wait_limit_ns)
        a.dy_stride = _stride(_match(dy, x, "dy"), "dy")
        a.dx_stride = C if out is None else _stride(_match(out, x, "out"), "out")
        sets = -(-T // rows_per_batch) if rows_per_batch else 1
        shape = ((sets, C) if rows_per_batch else (C,)) if weight is None else \
            (weight.shape if weight.dim() == 1 else (sets, C))
        plan = _keep(key, _Plan(a, load().qknr_ln_workspace_bytes, (shape, sets * C)))
    shape, n = plan.info
    if out is None:
        out = _empty(x.shape, x.dtype, x, stream)
    dweight = _empty(shape, torch.float32, x, stream) if dweight is None else _vector(dweight, n, "dweight", x)
    dbias = _empty(shape, torch.float32, x, stream) if dbias is None else _vector(dbias, n, "dbias", x)
    a = plan.new()
    a.x, a.dy, a.dx = x.data_ptr(), dy.data_ptr(), out.data_ptr()
    a.mean, a.rstd = _vector(mean, T, "mean", x).data_ptr(), _vector(rstd, T, "rstd", x).data_ptr()
    a.dweight, a.dbias = dweight.data_ptr(), dbias.data_ptr()
    if weight is not None:
        a.weight = weight.data_ptr()
    _status(a, status, dev_status, x)
    workspace = _workspace(a, plan, workspace, x, stream)
    _call((_lib or load()).qknr_ln_backward, a, stream, x)
    return out, dweight, dbias


# ---------------------------------------------------------------------------
# the root-mean-square norm with the residual's addition (include/qknr_rms.h)

def rms_args(x, weight=None, *, rows_per_batch=None, unit_offset=False, eps=1e-6, dev_status=None, flags=0,
             wait_limit_ns=0) -> QknrRmsArgs:
    """The arguments both passes share: token rows ``x`` [T, C] and ``weight``
    [C] or [B, C] (float32 or x's dtype; may be None), row t taking row
    t // rows_per_batch of it (default: one row)."""
    a = QknrRmsArgs()
    load().qknr_rms_args_init(ctypes.byref(a))
    if x.dtype not in _ACT:
        raise ValueError("x must be bfloat16 or float16")
    a.dtype = _ACT[x.dtype]
    a.x, a.x_stride = x.data_ptr(), _stride(x, "x")
    a.tokens, a.hidden = x.shape
    a.rows_per_batch = rows_per_batch or 0
    sets = -(-x.shape[0] // rows_per_batch) if rows_per_batch else 1
    if weight is not None:
        rows = weight.view(1, -1) if weight.dim() == 1 else weight
        if rows.dim() != 2 or rows.shape[1] != x.shape[1] or rows.shape[0] < sets:
            raise ValueError(f"weight must be [C] or [{sets}, C]")
        if weight.dtype not in (torch.float32, x.dtype):
            raise ValueError("weight must be float32 or of x's dtype")
        a.weight, a.param_stride = weight.data_ptr(), _stride(rows, "weight")
        a.param_dtype = FP32 if weight.dtype == torch.float32 else a.dtype
    a.eps = eps
    a.dev_status = _ptr(dev_status)
    a.flags, a.wait_limit_ns = flags | (RMS_UNIT_OFFSET if unit_offset else 0), wait_limit_ns
    return a


def _rms_forward(small, block, x, weight, residual, rows_per_batch, unit_offset, out, scales, sum_out, rstd, eps, stream,
                 status, dev_status, flags, wait_limit_ns):
    key = ("rms", small, block, _meta(x), _meta(weight), _meta(residual), _meta(out), _meta(sum_out), rows_per_batch,
           unit_offset, eps, flags, wait_limit_ns)
    plan = _plans.get(key)
    if plan is None:
        _one_device(x, weight, residual, out, sum_out)
        a = rms_args(x, weight, rows_per_batch=rows_per_batch, unit_offset=unit_offset, eps=eps, flags=flags,
                     wait_limit_ns=wait_limit_ns)
        if block not in (None, RMS_BLOCK) or (block and x.shape[1] % block):
            raise ValueError(f"block must be None or {RMS_BLOCK}, with as many columns or a multiple")
        shape = (x.shape[0], x.shape[1] // block) if block else (x.shape[0],)
        a.out, a.scale_block = RMS_OUT_E4M3 if small else RMS_OUT_SAME, block or 0
        if residual is not None:
            a.residual_stride = _stride(_match(residual, x, "residual"), "residual")
        elif sum_out is not None:
            raise ValueError("sum_out is the sum with a residual")
        if sum_out is not None:
            a.sum_stride = _stride(_match(sum_out, x, "sum_out"), "sum_out")
        if out is not None:
            if out.shape != x.shape or out.dtype != (torch.float8_e4m3fn if small else x.dtype):
                raise ValueError(f"out must be {tuple(x.shape)} of {torch.float8_e4m3fn if small else x.dtype}")
            a.y_stride = _stride(out, "out")
        plan = _keep(key, _Plan(a, None, (shape, math.prod(shape))))
    T = x.shape[0]
    if out is None:
        out = _empty(x.shape, torch.float8_e4m3fn if small else x.dtype, x, stream)
    rstd = _empty((T,), torch.float32, x, stream) if rstd is None else _vector(rstd, T, "rstd", x)
    a = plan.new()
    a.x, a.y, a.rstd = x.data_ptr(), out.data_ptr(), rstd.data_ptr()
    if weight is not None:
        a.weight = weight.data_ptr()
    if small:
        shape, n = plan.info
        scales = _empty(shape, torch.float32, x, stream) if scales is None else _vector(scales, n, "scales", x)
        a.scales = scales.data_ptr()
    h = x
    if residual is not None:
        h = _empty(x.shape, x.dtype, x, stream) if sum_out is None else sum_out
        a.residual, a.sum = residual.data_ptr(), h.data_ptr()
    _status(a, status, dev_status, x)
    _call((_lib or load()).qknr_rms_forward, a, stream, x)
    return out, scales, rstd, h


def rms_norm(x, weight=None, *, residual=None, rows_per_batch=None, unit_offset=False, out=None, sum_out=None, rstd=None,
             eps=1e-6, stream=None, status=True, dev_status=None, flags=0, wait_limit_ns=0):
    """Root-mean-square norm of token rows ``x`` [T, C], after the addition of
    ``residual`` (like x, or None): returns (y, rstd, h) with rstd float32 [T]
    and h = x + residual in x's dtype, the next residual (x itself without
    one).  h and rstd are what the backward pass needs.

    ``weight`` is [C], or [B, C] with row t taking row t // rows_per_batch;
    with ``unit_offset`` the gain is 1 + weight.  Results go to ``out`` (may be
    x, whose values are then gone where there is no residual) and ``sum_out``
    (may be residual or x), new tensors by default."""
    out, _, rstd, h = _rms_forward(False, None, x, weight, residual, rows_per_batch, unit_offset, out, None, sum_out, rstd,
                                   eps, stream, status, dev_status, flags, wait_limit_ns)
    return out, rstd, h


def rms_norm_quantized(x, weight=None, *, residual=None, block=None, rows_per_batch=None, unit_offset=False, out=None,
                       scales=None, sum_out=None, rstd=None, eps=1e-6, stream=None, status=True, dev_status=None, flags=0,
                       wait_limit_ns=0):
    """``rms_norm`` into 8 bits, the input of an 8-bit projection: returns
    (y, scales, rstd, h) with y torch.float8_e4m3fn [T, C] and scales float32
    [T], or with ``block=128`` [T, C / 128], so that y * scale is the norm."""
    return _rms_forward(True, block, x, weight, residual, rows_per_batch, unit_offset, out, scales, sum_out, rstd, eps,
                        stream, status, dev_status, flags, wait_limit_ns)


def rms_norm_backward(dy, x, weight, rstd, *, dsum=None, rows_per_batch=None, unit_offset=False, out=None, dweight=None,
                      workspace=None, stream=None, status=True, dev_status=None, flags=0, wait_limit_ns=0):
    """Gradients of ``rms_norm`` for its h as ``x``: returns (dx, dweight).  dx
    is the gradient of the forward pass's x and of its residual alike; ``dsum``,
    the gradient that reaches h past the norm, is added to it.  dweight is
    float32, [C] or a row for each sample (None without a weight).  ``out``
    receives dx (default: a new tensor; dy or dsum: in place)."""
    T, C = x.shape
    if T == 0 and weight is not None and weight.dim() == 1:
        rows_per_batch = None                     # no samples, but a gradient of the one row: zero
    key = ("rms_bwd", _meta(dy), _meta(x), _meta(weight), _meta(dsum), _meta(out), rows_per_batch, unit_offset, flags,
           wait_limit_ns)
    plan = _plans.get(key)
    if plan is None:
        _one_device(x, dy, weight, dsum, out)
        a = rms_args(x, weight, rows_per_batch=rows_per_batch, unit_offset=unit_offset, flags=flags,
                     wait_limit_ns=wait_limit_ns)
        a.dy_stride = _stride(_match(dy, x, "dy"), "dy")
        if dsum is not None:
            a.dsum_stride = _stride(_match(dsum, x, "dsum"), "dsum")
        if out is not None:
            a.dx_stride = _stride(_match(out, x, "out"), "out")
        sets = -(-T // rows_per_batch) if rows_per_batch else 1
        shape = (C,) if weight is None or weight.dim() == 1 else (sets, C)
        plan = _keep(key, _Plan(a, load().qknr_rms_workspace_bytes, (shape, math.prod(shape))))
    shape, n = plan.info
    if out is None:
        out = _empty(x.shape, x.dtype, x, stream)
    if weight is None:
        if dweight is not None:
            raise ValueError("dweight is the gradient of a weight")
    else:
        dweight = _empty(shape, torch.float32, x, stream) if dweight is None else _vector(dweight, n, "dweight", x)
    a = plan.new()
    a.x, a.dy, a.dx, a.rstd = x.data_ptr(), dy.data_ptr(), out.data_ptr(), _vector(rstd, T, "rstd", x).data_ptr()
    if weight is not None:
        a.weight, a.dweight = weight.data_ptr(), dweight.data_ptr()
    if dsum is not None:
        a.dsum = dsum.data_ptr()
    _status(a, status, dev_status, x)
    workspace = _workspace(a, plan, workspace, x, stream)
    _call((_lib or load()).qknr_rms_backward, a, stream, x)
    return out, dweight


# ---------------------------------------------------------------------------
# the backward pass of the fused QK-RMSNorm + RoPE (include/qknr_grad.h)

def grad_args(*, head_dim, q=None, k=None, dq=None, dk=None, dv=None, dq_out=None, dk_out=None, dv_out=None,
              n_heads_q=0, n_heads_k=0, n_heads_v=0, gamma_q=None, gamma_k=None, cos=None, sin=None,
              rope_style="interleaved", cos_layout="shared_row", cos_rows=None, eps=1e-6, tokens=0, dev_status=None,
              flags=0) -> QknrGradArgs:
    """Build a ``QknrGradArgs`` from tensors: q and k as the forward call got
    them, dq, dk and dv the gradients of its outputs."""
    a = QknrGradArgs()
    load().qknr_grad_args_init(ctypes.byref(a))
    acts = {"q": q, "k": k, "dq": dq, "dk": dk, "dv": dv, "dq_out": dq_out, "dk_out": dk_out, "dv_out": dv_out}
    given = [t for t in acts.values() if t is not None]
    if not given or given[0].dtype not in _ACT or any(t.dtype != given[0].dtype for t in given):
        raise ValueError("q, k and the gradients must share one dtype: bfloat16 or float16")
    a.dtype = _ACT[given[0].dtype]
    for name, t in acts.items():
        if t is None:
            continue
        heads = {"q": n_heads_q, "k": n_heads_k, "v": n_heads_v}[name.replace("_out", "")[-1]]
        stride = _stride(t, name)
        if t.shape != (tokens, heads * head_dim):
            raise ValueError(f"{name} must be [{tokens}, {heads * head_dim}]")
        setattr(a, name, t.data_ptr())
        setattr(a, name + "_stride", stride)
    a.tokens = tokens
    a.n_heads_q, a.n_heads_k, a.n_heads_v, a.head_dim = n_heads_q, n_heads_k, n_heads_v, head_dim
    for g, name in ((gamma_q, "gamma_q"), (gamma_k, "gamma_k")):
        if g is not None:
            setattr(a, name, _vector(g, head_dim, name).data_ptr())
    a.eps = eps
    if cos is not None:
        if cos.dtype not in _TAB or sin is None or sin.dtype != cos.dtype or cos.shape != sin.shape:
            raise ValueError("cos and sin must be of one shape, both float32 or both bfloat16")
        if not (cos.is_contiguous() and sin.is_contiguous() and cos.is_cuda and sin.is_cuda):
            raise ValueError("cos and sin must be contiguous CUDA tensors")
        a.cos_dtype = _TAB[cos.dtype]
        a.cos, a.sin = cos.data_ptr(), sin.data_ptr()
        a.cos_rows = cos.shape[0] if cos_rows is None else cos_rows
        if tokens and not 0 < a.cos_rows <= cos.shape[0]:
            raise ValueError("cos_rows must be between 1 and cos's rows")
    a.cos_layout = COS_LAYOUT[cos_layout]
    a.rope_style = ROPE[rope_style]
    a.dev_status = _ptr(dev_status)
    a.flags = flags
    return a


def qk_norm_rope_packed_backward(dout, qkv, n_heads_q, n_heads_k, n_heads_v, head_dim, gamma_q, gamma_k, cos, sin, *,
                                 out=None, rope_style="interleaved", cos_layout="shared_row", cos_rows=None, eps=1e-6,
                                 workspace=None, stream=None, status=True, dev_status=None, flags=0):
    """Backward pass of ``qk_norm_rope_packed``: ``qkv`` is that call's input
    (run it with ``out=``, so that the input survives), ``dout`` the gradient
    of its output.  Returns (dqkv, dgamma_q, dgamma_k), the gains' gradients
    float32 [head_dim] (None for a tensor without heads).  In place of
    ``dout`` unless ``out`` is given, which also receives a copy of V's
    gradient."""
    D = head_dim
    key = ("qk_bwd", _meta(dout), _meta(qkv), _meta(out), n_heads_q, n_heads_k, n_heads_v, D, _meta(gamma_q),
           _meta(gamma_k), _meta(cos), _meta(sin), rope_style, cos_layout, cos_rows, eps, flags)
    plan = _plans.get(key)
    k0, v0 = n_heads_q * D * 2, (n_heads_q + n_heads_k) * D * 2   # bytes into a row
    if plan is None:
        width = (n_heads_q + n_heads_k + n_heads_v) * D
        if qkv.dim() != 2 or qkv.shape[1] != width:
            raise ValueError(f"qkv must be [tokens, {width}]")
        _match(dout, qkv, "dout")
        if out is not None:
            _match(out, qkv, "out")
        _one_device(qkv, dout, out, gamma_q, gamma_k, cos, sin)
        _check_table(cos, D, cos_layout, n_heads_q or n_heads_k)

        def cols(t, a, b):
            return None if t is None or a == b else t[:, a // 2:b // 2]

        end = width * 2
        a = grad_args(q=cols(qkv, 0, k0), k=cols(qkv, k0, v0), dq=cols(dout, 0, k0), dk=cols(dout, k0, v0),
                      dv=cols(dout, v0, end), dq_out=cols(out, 0, k0), dk_out=cols(out, k0, v0),
                      dv_out=cols(out, v0, end), n_heads_q=n_heads_q, n_heads_k=n_heads_k, n_heads_v=n_heads_v,
                      head_dim=D, gamma_q=gamma_q if n_heads_q else None, gamma_k=gamma_k if n_heads_k else None,
                      cos=cos, sin=sin, rope_style=rope_style, cos_layout=cos_layout, cos_rows=cos_rows, eps=eps,
                      tokens=qkv.shape[0], flags=flags)
        plan = _keep(key, _Plan(a, load().qknr_grad_workspace_bytes))
    a = plan.new()
    x, d = qkv.data_ptr(), dout.data_ptr()
    o = d if out is None else out.data_ptr()
    dgq = dgk = None
    if n_heads_q:
        dgq = _empty((D,), torch.float32, qkv, stream)
        a.q, a.dq, a.dq_out, a.gamma_q, a.dgamma_q = x, d, o, gamma_q.data_ptr(), dgq.data_ptr()
    if n_heads_k:
        dgk = _empty((D,), torch.float32, qkv, stream)
        a.k, a.dk, a.dk_out, a.gamma_k, a.dgamma_k = x + k0, d + k0, o + k0, gamma_k.data_ptr(), dgk.data_ptr()
    if n_heads_v and out is not None:
        a.dv, a.dv_out = d + v0, o + v0
    a.cos, a.sin = cos.data_ptr(), sin.data_ptr()
    _status(a, status, dev_status, qkv)
    workspace = _workspace(a, plan, workspace, qkv, stream)
    _call((_lib or load()).qknr_backward, a, stream, qkv)
    return dout if out is None else out, dgq, dgk


def qk_norm_rope_tensor_backward(dout, x, n_heads, head_dim, gamma, cos, sin, *, out=None, rope_style="interleaved",
                                 cos_layout="shared_row", cos_rows=None, eps=1e-6, workspace=None, stream=None,
                                 status=True, dev_status=None, flags=0):
    """Backward pass of ``qk_norm_rope_tensor`` (one Q or K tensor [T, H*D]):
    returns (dx, dgamma).  In place of ``dout`` unless ``out`` is given."""
    dx, dgamma, _ = qk_norm_rope_packed_backward(dout, x, n_heads, 0, 0, head_dim, gamma, None, cos, sin, out=out,
                                                 rope_style=rope_style, cos_layout=cos_layout, cos_rows=cos_rows,
                                                 eps=eps, workspace=workspace, stream=stream, status=status,
                                                 dev_status=dev_status, flags=flags)
    return dx, dgamma


# ---------------------------------------------------------------------------
# attention and its backward pass (include/qknr_attn.h)

def attn_args(q, k, v, n_heads_q, n_heads_k, head_dim, *, batch=1, scale=None, causal=False, q_lens=None, k_lens=None,
              dev_status=None, flags=0, wait_limit_ns=0) -> QknrAttnArgs:
    """The arguments both passes share: token rows q [batch * seq_q, Hq * D],
    k and v [batch * seq_k, Hk * D] (views with any row stride, such as the
    columns of a packed QKV activation)."""
    a = QknrAttnArgs()
    load().qknr_attn_args_init(ctypes.byref(a))
    if q.dtype not in _ACT or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v must share one dtype: bfloat16 or float16")
    a.dtype = _ACT[q.dtype]
    for name, t, heads in (("q", q, n_heads_q), ("k", k, n_heads_k), ("v", v, n_heads_k)):
        setattr(a, name + "_stride", _stride(t, name))
        if t.dim() != 2 or t.shape[1] != heads * head_dim or batch < 1 or t.shape[0] % batch:
            raise ValueError(f"{name} must be [batch * seq, {heads * head_dim}]")
        setattr(a, name, t.data_ptr())
    if k.shape[0] != v.shape[0]:
        raise ValueError("k and v need the same number of rows")
    a.batch, a.seq_q, a.seq_k = batch, q.shape[0] // batch, k.shape[0] // batch
    a.n_heads_q, a.n_heads_k, a.head_dim = n_heads_q, n_heads_k, head_dim
    for name, t in (("q_lens", q_lens), ("k_lens", k_lens)):
        if t is not None:
            if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous() or t.numel() != batch:
                raise ValueError(f"{name} must be a contiguous int32 CUDA tensor of {batch} values")
            setattr(a, name, t.data_ptr())
    if scale is not None:
        a.scale = scale
        if not 0 < a.scale < float("inf"):                  # as fp32
            raise ValueError("scale must be positive and finite")
    a.causal = int(bool(causal))
    a.dev_status = _ptr(dev_status)
    a.flags, a.wait_limit_ns = flags, wait_limit_ns
    return a


def attention(q, k, v, n_heads_q, n_heads_k, head_dim, *, batch=1, scale=None, causal=False, q_lens=None, k_lens=None,
              out=None, lse=None, workspace=None, stream=None, status=True, dev_status=None, flags=0, wait_limit_ns=0):
    """Attention over token rows: returns (o [batch * seq_q, Hq * D], lse
    float32 [batch, Hq, seq_q]).  ``q_lens``/``k_lens`` (int32 [batch] on the
    device) end each sample's queries and keys, ``causal`` lines the diagonal
    up with their last ones; a query that sees no key answers zero with lse
    -inf.  ``out`` and ``lse`` receive the results (default: new tensors)."""
    key = ("attn", _meta(q), _meta(k), _meta(v), n_heads_q, n_heads_k, head_dim, batch, scale, causal, _meta(q_lens),
           _meta(k_lens), _meta(out), flags, wait_limit_ns)
    plan = _plans.get(key)
    if plan is None:
        _one_device(q, k, v, q_lens, k_lens, out)
        a = attn_args(q, k, v, n_heads_q, n_heads_k, head_dim, batch=batch, scale=scale, causal=causal, q_lens=q_lens,
                      k_lens=k_lens, flags=flags, wait_limit_ns=wait_limit_ns)
        a.o_stride = 0 if out is None else _stride(_match(out, q, "out"), "out")
        plan = _keep(key, _Plan(a, load().qknr_attn_workspace_bytes, ((batch, n_heads_q, a.seq_q), q.shape[0] * n_heads_q)))
    shape, n = plan.info
    if out is None:
        out = _empty(q.shape, q.dtype, q, stream)
    lse = _empty(shape, torch.float32, q, stream) if lse is None else _vector(lse, n, "lse", q)
    a = plan.new()
    a.q, a.k, a.v, a.o, a.lse = q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr()
    if q_lens is not None:
        a.q_lens = q_lens.data_ptr()
    if k_lens is not None:
        a.k_lens = k_lens.data_ptr()
    _status(a, status, dev_status, q)
    workspace = _workspace(a, plan, workspace, q, stream)
    _call((_lib or load()).qknr_attn_forward, a, stream, q)
    return out, lse


def attention_backward(do, q, k, v, o, lse, n_heads_q, n_heads_k, head_dim, *, batch=1, scale=None, causal=False,
                       q_lens=None, k_lens=None, dq=None, dk=None, dv=None, workspace=None, stream=None, status=True,
                       dev_status=None, flags=0, wait_limit_ns=0):
    """Gradients of ``attention`` from do, its inputs and its outputs o and
    lse: returns (dq, dk, dv), new tensors unless given (column views of one
    packed buffer are fine).  Rows past the lengths get zero."""
    key = ("attn_bwd", _meta(do), _meta(q), _meta(k), _meta(v), _meta(o), n_heads_q, n_heads_k, head_dim, batch, scale,
           causal, _meta(q_lens), _meta(k_lens), _meta(dq), _meta(dk), _meta(dv), flags, wait_limit_ns)
    plan = _plans.get(key)
    if plan is None:
        _one_device(q, do, k, v, o, q_lens, k_lens, dq, dk, dv)
        a = attn_args(q, k, v, n_heads_q, n_heads_k, head_dim, batch=batch, scale=scale, causal=causal, q_lens=q_lens,
                      k_lens=k_lens, flags=flags, wait_limit_ns=wait_limit_ns)
        a.o_stride, a.dout_stride = _stride(_match(o, q, "o"), "o"), _stride(_match(do, q, "do"), "do")
        for name, t, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
            if t is not None:
                setattr(a, name + "_stride", _stride(_match(t, like, name), name))
        plan = _keep(key, _Plan(a, load().qknr_attn_backward_workspace_bytes, q.shape[0] * n_heads_q))
    if dq is None:
        dq = _empty(q.shape, q.dtype, q, stream)
    if dk is None:
        dk = _empty(k.shape, k.dtype, k, stream)
    if dv is None:
        dv = _empty(v.shape, v.dtype, v, stream)
    a = plan.new()
    a.q, a.k, a.v, a.o, a.dout = q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr()
    a.lse = _vector(lse, plan.info, "lse", q).data_ptr()
    a.dq, a.dk, a.dv = dq.data_ptr(), dk.data_ptr(), dv.data_ptr()
    if q_lens is not None:
        a.q_lens = q_lens.data_ptr()
    if k_lens is not None:
        a.k_lens = k_lens.data_ptr()
    _status(a, status, dev_status, q)
    workspace = _workspace(a, plan, workspace, q, stream)
    _call((_lib or load()).qknr_attn_backward, a, stream, q)
    return dq, dk, dv


# ---------------------------------------------------------------------------
# attention over packed sequences and its backward pass (include/qknr_pack.h)

def _int32s(t, n, name):
    if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous() or t.numel() != n:
        raise ValueError(f"{name} must be a contiguous int32 CUDA tensor of {n} values")
    return t.data_ptr()


def _heads_of(a, tensors, n_heads_q, n_heads_k, head_dim):
    """The types, widths and strides of q, k, v and tensors like them into a."""
    first = next(t for _, t in tensors)
    if first.dtype not in _ACT or any(t.dtype != first.dtype for _, t in tensors):
        raise ValueError(", ".join(name for name, _ in tensors) + " must share one dtype: bfloat16 or float16")
    a.dtype = _ACT[first.dtype]
    a.n_heads_q, a.n_heads_k, a.head_dim = n_heads_q, n_heads_k, head_dim
    for name, t in tensors:
        heads = n_heads_q if name == "q" else n_heads_k
        setattr(a, name + "_stride", _stride(t, name))
        if t.shape[1] != heads * head_dim:
            raise ValueError(f"{name} must be [rows, {heads * head_dim}]")
        setattr(a, name, t.data_ptr())


def _scale_of(a, scale):
    if scale is not None:
        a.scale = scale
        if not 0 < a.scale < float("inf"):                  # as fp32
            raise ValueError("scale must be positive and finite")


def pack_args(q, k, v, n_heads_q, n_heads_k, head_dim, q_starts, k_starts=None, *, scale=None, causal=False, dev_status=None,
              flags=0, wait_limit_ns=0) -> QknrPackArgs:
    """The arguments both passes share: token rows q [rows_q, Hq * D], k and v
    [rows_k, Hk * D] (views with any row stride) and where the sequences begin
    in them (int32 [batch + 1] on the device; ``k_starts`` None: q_starts)."""
    a = QknrPackArgs()
    load().qknr_pack_args_init(ctypes.byref(a))
    _heads_of(a, (("q", q), ("k", k), ("v", v)), n_heads_q, n_heads_k, head_dim)
    if k.shape[0] != v.shape[0]:
        raise ValueError("k and v need the same number of rows")
    if max(q.shape[0], k.shape[0]) >= 1 << 31:
        raise ValueError("2^31 rows or more")
    a.rows_q, a.rows_k, a.batch = q.shape[0], k.shape[0], max(q_starts.numel() - 1, 0)
    a.q_starts = _int32s(q_starts, a.batch + 1, "q_starts")
    if k_starts is not None:
        a.k_starts = _int32s(k_starts, a.batch + 1, "k_starts")
    _scale_of(a, scale)
    a.causal = int(bool(causal))
    a.dev_status = _ptr(dev_status)
    a.flags, a.wait_limit_ns = flags, wait_limit_ns
    return a


def attention_packed(q, k, v, n_heads_q, n_heads_k, head_dim, q_starts, k_starts=None, *, scale=None, causal=False, out=None,
                     lse=None, workspace=None, stream=None, status=True, dev_status=None, flags=0, wait_limit_ns=0):
    """Attention over sequences packed one after the other: sequence b is the
    rows q_starts[b] .. q_starts[b + 1] - 1 of q [rows_q, Hq * D] and
    k_starts[b] .. of k and v [rows_k, Hk * D] (int32 [batch + 1] on the device;
    ``k_starts`` None: q_starts).  Returns (o [rows_q, Hq * D], lse float32
    [Hq, rows_q]); ``causal`` and what a query without keys answers are
    ``attention``'s.  Rows that belong to no sequence keep what ``out`` and
    ``lse`` held there (new tensors by default, uninitialised)."""
    key = ("pack", _meta(q), _meta(k), _meta(v), n_heads_q, n_heads_k, head_dim, _meta(q_starts), _meta(k_starts), scale,
           causal, _meta(out), flags, wait_limit_ns)
    plan = _plans.get(key)
    if plan is None:
        _one_device(q, k, v, q_starts, k_starts, out)
        a = pack_args(q, k, v, n_heads_q, n_heads_k, head_dim, q_starts, k_starts, scale=scale, causal=causal, flags=flags,
                      wait_limit_ns=wait_limit_ns)
        a.o_stride = 0 if out is None else _stride(_match(out, q, "out"), "out")
        plan = _keep(key, _Plan(a, load().qknr_pack_workspace_bytes))
    if out is None:
        out = _empty(q.shape, q.dtype, q, stream)
    n = q.shape[0] * n_heads_q
    lse = _empty((n_heads_q, q.shape[0]), torch.float32, q, stream) if lse is None else _vector(lse, n, "lse", q)
    a = plan.new()
    a.q, a.k, a.v, a.o, a.lse = q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr()
    a.q_starts = q_starts.data_ptr()
    if k_starts is not None:
        a.k_starts = k_starts.data_ptr()
    _status(a, status, dev_status, q)
    workspace = _workspace(a, plan, workspace, q, stream)
    _call((_lib or load()).qknr_pack_forward, a, stream, q)
    return out, lse


def attention_packed_backward(do, q, k, v, o, lse, n_heads_q, n_heads_k, head_dim, q_starts, k_starts=None, *, scale=None,
                              causal=False, dq=None, dk=None, dv=None, workspace=None, stream=None, status=True,
                              dev_status=None, flags=0, wait_limit_ns=0):
    """Gradients of ``attention_packed`` from do, its inputs and its outputs o
    and lse: returns (dq, dk, dv), new tensors unless given (column views of
    one packed buffer are fine).  With o and lse over more keys than the call
    has (keys split over calls) they are its keys' part.  Rows that belong to
    no sequence keep what they held."""
    key = ("pack_bwd", _meta(do), _meta(q), _meta(k), _meta(v), _meta(o), n_heads_q, n_heads_k, head_dim, _meta(q_starts),
           _meta(k_starts), scale, causal, _meta(dq), _meta(dk), _meta(dv), flags, wait_limit_ns)
    plan = _plans.get(key)
    if plan is None:
        _one_device(q, do, k, v, o, q_starts, k_starts, dq, dk, dv)
        a = pack_args(q, k, v, n_heads_q, n_heads_k, head_dim, q_starts, k_starts, scale=scale, causal=causal, flags=flags,
                      wait_limit_ns=wait_limit_ns)
        a.o_stride, a.dout_stride = _stride(_match(o, q, "o"), "o"), _stride(_match(do, q, "do"), "do")
        for name, t, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
            if t is not None:
                setattr(a, name + "_stride", _stride(_match(t, like, name), name))
        plan = _keep(key, _Plan(a, load().qknr_pack_backward_workspace_bytes))
    if dq is None:
        dq = _empty(q.shape, q.dtype, q, stream)
    if dk is None:
        dk = _empty(k.shape, k.dtype, k, stream)
    if dv is None:
        dv = _empty(v.shape, v.dtype, v, stream)
    a = plan.new()
    a.q, a.k, a.v, a.o, a.dout = q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr()
    a.lse = _vector(lse, q.shape[0] * n_heads_q, "lse", q).data_ptr()
    a.dq, a.dk, a.dv = dq.data_ptr(), dk.data_ptr(), dv.data_ptr()
    a.q_starts = q_starts.data_ptr()
    if k_starts is not None:
        a.k_starts = k_starts.data_ptr()
    _status(a, status, dev_status, q)
    workspace = _workspace(a, plan, workspace, q, stream)
    _call((_lib or load()).qknr_pack_backward, a, stream, q)
    return dq, dk, dv


# ---------------------------------------------------------------------------
# attention beside a shared prefix (include/qknr_prefix.h)

def prefix_args(q, k, v, prefix_k, prefix_v, n_heads_q, n_heads_k, head_dim, *, batch=1, scale=None, causal=False,
                q_lens=None, k_lens=None, dev_status=None, flags=0, wait_limit_ns=0) -> QknrPrefixArgs:
    """The arguments of ``attention_prefix`` without its outputs."""
    a = QknrPrefixArgs()
    load().qknr_prefix_args_init(ctypes.byref(a))
    _heads_of(a, (("q", q), ("k", k), ("v", v), ("prefix_k", prefix_k), ("prefix_v", prefix_v)), n_heads_q, n_heads_k, head_dim)
    if batch < 1 or q.shape[0] % batch or k.shape[0] % batch:
        raise ValueError("q, k and v must be [batch * seq, ...]")
    if k.shape[0] != v.shape[0] or prefix_k.shape[0] != prefix_v.shape[0]:
        raise ValueError("k and v, prefix_k and prefix_v need the same number of rows")
    if max(q.shape[0], k.shape[0], prefix_k.shape[0]) >= 1 << 31:
        raise ValueError("2^31 rows or more")
    a.batch, a.seq_q, a.seq_k, a.prefix = batch, q.shape[0] // batch, k.shape[0] // batch, prefix_k.shape[0]
    for name, t in (("q_lens", q_lens), ("k_lens", k_lens)):
        if t is not None:
            setattr(a, name, _int32s(t, batch, name))
    _scale_of(a, scale)
    a.causal = int(bool(causal))
    a.dev_status = _ptr(dev_status)
    a.flags, a.wait_limit_ns = flags, wait_limit_ns
    return a


def attention_prefix(q, k, v, prefix_k, prefix_v, n_heads_q, n_heads_k, head_dim, *, batch=1, scale=None, causal=False,
                     q_lens=None, k_lens=None, out=None, lse=None, workspace=None, stream=None, status=True, dev_status=None,
                     flags=0, wait_limit_ns=0):
    """``attention`` for samples whose keys all begin with the same rows
    ``prefix_k`` and ``prefix_v`` [prefix, Hk * D], held once: query rows q
    [batch * seq_q, Hq * D] see all of the prefix and, as in ``attention``,
    their sample's own k and v [batch * seq_k, Hk * D] (seq_k may be 0).
    Returns (o, lse float32 [batch, Hq, seq_q]) over both."""
    key = ("prefix", _meta(q), _meta(k), _meta(v), _meta(prefix_k), _meta(prefix_v), n_heads_q, n_heads_k, head_dim, batch,
           scale, causal, _meta(q_lens), _meta(k_lens), _meta(out), flags, wait_limit_ns)
    plan = _plans.get(key)
    if plan is None:
        _one_device(q, k, v, prefix_k, prefix_v, q_lens, k_lens, out)
        a = prefix_args(q, k, v, prefix_k, prefix_v, n_heads_q, n_heads_k, head_dim, batch=batch, scale=scale, causal=causal,
                        q_lens=q_lens, k_lens=k_lens, flags=flags, wait_limit_ns=wait_limit_ns)
        a.o_stride = 0 if out is None else _stride(_match(out, q, "out"), "out")
        plan = _keep(key, _Plan(a, load().qknr_prefix_workspace_bytes, ((batch, n_heads_q, a.seq_q), q.shape[0] * n_heads_q)))
    shape, n = plan.info
    if out is None:
        out = _empty(q.shape, q.dtype, q, stream)
    lse = _empty(shape, torch.float32, q, stream) if lse is None else _vector(lse, n, "lse", q)
    a = plan.new()
    a.q, a.k, a.v, a.o, a.lse = q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr()
    a.prefix_k, a.prefix_v = prefix_k.data_ptr(), prefix_v.data_ptr()
    if q_lens is not None:
        a.q_lens = q_lens.data_ptr()
    if k_lens is not None:
        a.k_lens = k_lens.data_ptr()
    _status(a, status, dev_status, q)
    workspace = _workspace(a, plan, workspace, q, stream)
    _call((_lib or load()).qknr_prefix_forward, a, stream, q)
    return out, lse
