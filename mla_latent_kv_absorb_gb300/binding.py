"""ctypes binding of libmla_gb300.so: the C ABI of include/mla.h under the same names.

Argument marshalling only: torch tensors supply device memory and streams, every step of the
decode runs in the library's CUDA kernels.  If the library has not been built this module
raises; there is no fallback path.
"""
from __future__ import annotations

import ctypes
import math
import os
from contextlib import nullcontext
from functools import partial
from typing import Optional

import numpy as np
import torch

from . import D_C, D_HC, D_R, D_ROW, NUM_HEADS, PAGE

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmla_gb300.so")

# mla_status
MLA_OK, MLA_ERR_INVALID_ARG, MLA_ERR_ALIGNMENT, MLA_ERR_UNSUPPORTED = 0, 1, 2, 3
MLA_ERR_WORKSPACE, MLA_ERR_CUDA, MLA_ERR_DEVICE_FAULT = 4, 5, 6
# mla_kv_dtype
MLA_KV_BF16, MLA_KV_FP8_E4M3, MLA_KV_NVFP4 = 0, 1, 2
NVFP4_ROW = D_C // 2 + D_C // 16  # bytes of one token's NVFP4 row: packed e2m1 codes, then e4m3 block scales
# mla_dtype, mla_rope_layout, mla_rope_scaling, mla_w4_format
_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_ROPE_LAYOUTS = {"interleaved": 0, "half": 1}
_ROPE_SCALINGS = {"none": 0, "linear": 1, "yarn": 2}
MLA_ROPE_MAX_DIM = 256
MLA_W4_INT4, MLA_W4_NVFP4 = 0, 1
# device error bits
MLA_DEVERR_BAD_PAGE, MLA_DEVERR_TIMEOUT, MLA_DEVERR_SMEM_ALIGN, MLA_DEVERR_BAD_PLAN = 1, 2, 4, 8

SOFTMAX_SCALE = 1.0 / math.sqrt(D_HC + D_R)


class MlaError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn} failed: {msg} (status {status})")
        self.status = status


class PlanOptions(ctypes.Structure):
    _fields_ = [("min_pages_per_split", ctypes.c_int32), ("max_clusters", ctypes.c_int32),
                ("wait_timeout_ns", ctypes.c_int64), ("item_cost_pages", ctypes.c_int32),
                ("queries_per_seq", ctypes.c_int32), ("window", ctypes.c_int32), ("sinks", ctypes.c_int32)]


class PlanInfo(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("num_clusters", ctypes.c_int32), ("num_items", ctypes.c_int32),
                ("num_partials", ctypes.c_int32), ("num_combine", ctypes.c_int32), ("max_splits", ctypes.c_int32),
                ("total_pages", ctypes.c_int32), ("queries_per_seq", ctypes.c_int32), ("plan_bytes", ctypes.c_int64),
                ("workspace_bytes", ctypes.c_int64), ("wait_timeout_ns", ctypes.c_int64), ("window", ctypes.c_int32),
                ("sinks", ctypes.c_int32)]


EXPORTS = ("mla_status_string", "mla_last_error_string", "mla_plan_bytes_max", "mla_plan_splits", "mla_absorb_q", "mla_decode_paged",
           "mla_combine_splits", "mla_out_proj", "mla_read_device_error", "mla_debug_wait_timeout",
           "mla_decode_paged_static_ws", "mla_decode_step_host", "mla_append_kv", "mla_merge_out_proj",
           "mla_absorb_decode_paged", "mla_gather_kv", "mla_step_graph_create", "mla_step_graph_run",
           "mla_step_graph_destroy", "mla_prefill_workspace_bytes", "mla_prefill_decompressed",
           "mla_rope_init", "mla_rope", "mla_rope_append_kv", "mla_w4_packed_bytes", "mla_w4_pack",
           "mla_linear_w4", "mla_absorb_q_w4", "mla_out_proj_w4", "mla_prefix_open", "mla_prefix_attend_workspace_bytes",
           "mla_prefix_attend", "mla_prefill_window_workspace_bytes", "mla_prefill_window", "mla_abi_version")

# of the header that the structures and signatures here restate
MLA_ABI_VERSION = 2

# capacity of the library's fixed split-partial array (mla_decode_paged_static_ws)
MLA_STATIC_WS_MAX_PARTIALS = 128

_lib = None


class StepBuffers(ctypes.Structure):
    """mla_step_buffers: the device buffers of mla_decode_step_host, plus its pinned plan staging."""
    _fields_ = [("q_c", ctypes.c_void_p), ("q_r", ctypes.c_void_p), ("q_abs", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("plan", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t), ("o_lat", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("out", ctypes.c_void_p), ("dev_error", ctypes.c_void_p), ("plan_host", ctypes.c_void_p),
                ("plan_capacity", ctypes.c_size_t)]


class RopeOptions(ctypes.Structure):
    _fields_ = [("dim", ctypes.c_int32), ("layout", ctypes.c_int32), ("scaling", ctypes.c_int32),
                ("original_len", ctypes.c_int32), ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("beta_fast", ctypes.c_double), ("beta_slow", ctypes.c_double), ("magnitude", ctypes.c_double),
                ("inv_freq", ctypes.c_void_p)]


class RopeConfig(ctypes.Structure):
    _fields_ = [("dim", ctypes.c_int32), ("layout", ctypes.c_int32), ("magnitude", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("step", ctypes.c_uint64 * (MLA_ROPE_MAX_DIM // 2))]


class W4Struct(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("heads", ctypes.c_int32), ("n", ctypes.c_int32), ("k", ctypes.c_int32),
                ("group", ctypes.c_int32), ("has_zero", ctypes.c_int32), ("tensor_scale", ctypes.c_float),
                ("packed", ctypes.c_void_p)]


def lib() -> ctypes.CDLL:
    """Open libmla_gb300.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() or "
                           "python -m mla_latent_kv_absorb_gb300.build")
    L = ctypes.CDLL(LIB_PATH)
    version = L.mla_abi_version() if hasattr(L, "mla_abi_version") else 1
    if version != MLA_ABI_VERSION:
        raise RuntimeError(f"{LIB_PATH} has ABI version {version}, this binding {MLA_ABI_VERSION}: build it again")
    P, i32, i64, sz, u32p = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p
    L.mla_status_string.restype = ctypes.c_char_p
    L.mla_status_string.argtypes = [ctypes.c_int]
    L.mla_last_error_string.restype = ctypes.c_char_p
    L.mla_last_error_string.argtypes = []
    L.mla_plan_bytes_max.restype = sz
    L.mla_plan_bytes_max.argtypes = [i32, i32]
    L.mla_plan_splits.restype = ctypes.c_int
    L.mla_plan_splits.argtypes = [P, i32, i32, ctypes.POINTER(PlanOptions), P, sz, ctypes.POINTER(PlanInfo)]
    L.mla_absorb_q.restype = ctypes.c_int
    L.mla_absorb_q.argtypes = [P, P, P, i32, P]
    L.mla_decode_paged.restype = ctypes.c_int
    L.mla_decode_paged.argtypes = [ctypes.POINTER(PlanInfo), P, P, P, ctypes.c_int, P, P, P, i32, P, i32,
                                   ctypes.c_float, P, sz, P, P, u32p, P]
    L.mla_decode_paged_static_ws.restype = ctypes.c_int
    L.mla_decode_paged_static_ws.argtypes = [ctypes.POINTER(PlanInfo), P, P, P, ctypes.c_int, P, P, P, i32, P, i32,
                                             ctypes.c_float, P, P, u32p, P]
    L.mla_combine_splits.restype = ctypes.c_int
    L.mla_combine_splits.argtypes = [ctypes.POINTER(PlanInfo), P, P, sz, P, P, P]
    L.mla_out_proj.restype = ctypes.c_int
    L.mla_out_proj.argtypes = [P, P, P, i32, P]
    L.mla_absorb_decode_paged.restype = ctypes.c_int
    L.mla_absorb_decode_paged.argtypes = [ctypes.POINTER(PlanInfo), P, P, P, P, P, P, ctypes.c_int, P, P, P, i32, P,
                                          i32, ctypes.c_float, P, sz, P, P, P, P]
    L.mla_gather_kv.restype = ctypes.c_int
    L.mla_gather_kv.argtypes = [ctypes.c_int, P, P, P, i32, P, i32, P, P, i32, P, P, P]
    L.mla_merge_out_proj.restype = ctypes.c_int
    L.mla_merge_out_proj.argtypes = [ctypes.POINTER(PlanInfo), P, P, sz, P, P, P, P, P, P]
    L.mla_decode_step_host.restype = ctypes.c_int
    L.mla_decode_step_host.argtypes = [P, i32, i32, ctypes.POINTER(PlanOptions), P, P, P, i32, P, P, ctypes.c_int, P,
                                       P, P, i32, ctypes.c_float, ctypes.POINTER(StepBuffers), P,
                                       ctypes.POINTER(PlanInfo), P]
    step_args = [P, i32, i32, ctypes.POINTER(PlanOptions), P, P, P, i32, P, P, ctypes.c_int, P, P, P, i32,
                 ctypes.c_float, ctypes.POINTER(StepBuffers), P, ctypes.POINTER(PlanInfo), P]
    L.mla_step_graph_create.restype = ctypes.c_int
    L.mla_step_graph_create.argtypes = step_args + [ctypes.POINTER(ctypes.c_void_p)]
    L.mla_step_graph_run.restype = ctypes.c_int
    L.mla_step_graph_run.argtypes = [P, i32, P]
    L.mla_step_graph_destroy.restype = ctypes.c_int
    L.mla_step_graph_destroy.argtypes = [P]
    L.mla_prefill_workspace_bytes.restype = sz
    L.mla_prefill_workspace_bytes.argtypes = [i32]
    L.mla_prefill_decompressed.restype = ctypes.c_int
    L.mla_prefill_decompressed.argtypes = [ctypes.c_int, P, P, P, i32, P, i32, i32, i32, P, P, P, P, ctypes.c_float,
                                           P, sz, P, u32p, P]
    L.mla_append_kv.restype = ctypes.c_int
    L.mla_append_kv.argtypes = [i32, P, P, P, ctypes.c_int, i32, P, P, P, u32p, P]
    L.mla_rope_init.restype = ctypes.c_int
    L.mla_rope_init.argtypes = [P, P]
    L.mla_rope.restype = ctypes.c_int
    L.mla_rope.argtypes = [P, ctypes.c_int, i32, i32, i32, i32, P, i64, i64, P, i64, i64, P, i64, i64, P, P]
    L.mla_rope_append_kv.restype = ctypes.c_int
    L.mla_rope_append_kv.argtypes = [P, i32, P, i64, P, i64, P, P, ctypes.c_int, i32, P, P, P, P, i64, i64, P, P, P, P]
    L.mla_w4_packed_bytes.restype = sz
    L.mla_w4_packed_bytes.argtypes = [P]
    L.mla_w4_pack.restype = ctypes.c_int
    L.mla_w4_pack.argtypes = [P, P, P, P, P, P]
    L.mla_linear_w4.restype = ctypes.c_int
    L.mla_linear_w4.argtypes = [i32, P, i64, i64, P, P, i64, i64, P]
    L.mla_absorb_q_w4.restype = ctypes.c_int
    L.mla_absorb_q_w4.argtypes = [P, P, P, i32, P]
    L.mla_out_proj_w4.restype = ctypes.c_int
    L.mla_out_proj_w4.argtypes = [P, P, P, i32, P]
    f32 = ctypes.c_float
    L.mla_prefix_open.restype = ctypes.c_int
    L.mla_prefix_open.argtypes = [ctypes.c_int, P, P, P, i32, P, i32, i32, P, P, P, P, P, P, P]
    L.mla_prefix_attend_workspace_bytes.restype = sz
    L.mla_prefix_attend_workspace_bytes.argtypes = [i32, i32, i32]
    L.mla_prefix_attend.restype = ctypes.c_int
    L.mla_prefix_attend.argtypes = [i32, i32, i32, P, P, P, P, P, i64, f32, P, P, P, sz, P, P, P, P]
    L.mla_prefill_window_workspace_bytes.restype = sz
    L.mla_prefill_window_workspace_bytes.argtypes = [i32, i32, i32, i32]
    L.mla_prefill_window.restype = ctypes.c_int
    L.mla_prefill_window.argtypes = [ctypes.c_int, P, P, P, i32, P, i32, i32, i32, i32, i32, P, P, P, P, f32, P, sz, P,
                                     P, P]
    L.mla_read_device_error.restype = ctypes.c_int
    L.mla_read_device_error.argtypes = [u32p, ctypes.POINTER(ctypes.c_uint32), P]
    L.mla_debug_wait_timeout.restype = ctypes.c_int
    L.mla_debug_wait_timeout.argtypes = [u32p, i64, P]
    _lib = L
    return L


def status_string(status: int) -> str:
    return lib().mla_status_string(int(status)).decode()


def _check(fn: str, status: int) -> None:
    if status != MLA_OK:
        msg = status_string(status)
        if status == MLA_ERR_CUDA or (status == MLA_ERR_WORKSPACE and fn == "mla_decode_paged_static_ws"):
            msg += ": " + lib().mla_last_error_string().decode()
        raise MlaError(fn, status, msg)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _addr(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else int(t.data_ptr())


def _stream(stream):
    if stream is None:  # the current stream's handle, without making a torch.cuda.Stream of it
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _need(t: torch.Tensor, name: str, dtype, shape=None, device=True):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if device and not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


def _i32(x) -> int:
    """A size for the C side, whose sizes have 32 bits: beyond them the nearest that they hold, not one that
    wrapped round.  What is too small is refused there; a window or sinks past every length are those."""
    return max(-1, min(int(x), 2 ** 31 - 1))


# --------------------------------------------------------------------------- C ABI, same names

def mla_plan_splits(seq_lens, num_sms: int, *, min_pages_per_split: int = 0, max_clusters: int = 0,
                    wait_timeout_ns: int = 0, item_cost_pages: int = 0, queries_per_seq: int = 0, window: int = 0,
                    sinks: int = 0):
    """Host planning. Returns (plan image as an int32 numpy array, PlanInfo).  With
    queries_per_seq = q > 1 the plan covers len(seq_lens) * q query rows (token t of sequence b
    is row b * q + t and sees the first S_b - q + 1 + t cached tokens); with window = W > 0 a row
    sees the last W of its tokens and the first ``sinks``."""
    lens = np.ascontiguousarray(np.asarray(seq_lens, dtype=np.int32))
    B = int(lens.size)
    cap = int(lib().mla_plan_bytes_max(B * max(1, int(queries_per_seq)), int(num_sms)))
    if cap == 0:
        raise MlaError("mla_plan_splits", MLA_ERR_INVALID_ARG, "bad batch or SM count")
    buf = np.zeros(cap // 4, dtype=np.int32)
    opts = PlanOptions(int(min_pages_per_split), int(max_clusters), int(wait_timeout_ns), int(item_cost_pages),
                       int(queries_per_seq), _i32(window), _i32(sinks))
    info = PlanInfo()
    st = lib().mla_plan_splits(lens.ctypes.data_as(ctypes.c_void_p), B, int(num_sms), ctypes.byref(opts),
                               buf.ctypes.data_as(ctypes.c_void_p), cap, ctypes.byref(info))
    _check("mla_plan_splits", st)
    return buf[: info.plan_bytes // 4].copy(), info


def mla_absorb_q(q_c: torch.Tensor, w_uk: torch.Tensor, q_abs: torch.Tensor, stream=None) -> None:
    B = q_c.shape[0]
    _need(q_c, "q_c", torch.bfloat16, (B, NUM_HEADS, D_HC))
    _need(w_uk, "w_uk", torch.bfloat16, (NUM_HEADS, D_HC, D_C))
    _need(q_abs, "q_abs", torch.bfloat16, (B, NUM_HEADS, D_C))
    _check("mla_absorb_q", lib().mla_absorb_q(_ptr(q_c), _ptr(w_uk), _ptr(q_abs), B, _stream(stream)))


def mla_out_proj(o_lat: torch.Tensor, w_uv: torch.Tensor, out: torch.Tensor, stream=None) -> None:
    B = o_lat.shape[0]
    _need(o_lat, "o_lat", torch.bfloat16, (B, NUM_HEADS, D_C))
    _need(w_uv, "w_uv", torch.bfloat16, (NUM_HEADS, D_HC, D_C))
    _need(out, "out", torch.bfloat16, (B, NUM_HEADS, D_HC))
    _check("mla_out_proj", lib().mla_out_proj(_ptr(o_lat), _ptr(w_uv), _ptr(out), B, _stream(stream)))


def mla_decode_paged(info: PlanInfo, plan_dev: torch.Tensor, q_abs: torch.Tensor, q_r: torch.Tensor, *,
                     kv_pool: torch.Tensor, block_table: torch.Tensor, o_lat: torch.Tensor, lse: torch.Tensor,
                     dev_error: torch.Tensor, workspace: Optional[torch.Tensor] = None,
                     kv_scale: Optional[torch.Tensor] = None, kr_pool: Optional[torch.Tensor] = None,
                     softmax_scale: float = SOFTMAX_SCALE, stream=None) -> None:
    B = q_abs.shape[0]
    _need(plan_dev, "plan_dev", torch.int32)
    _need(q_abs, "q_abs", torch.bfloat16, (B, NUM_HEADS, D_C))
    _need(q_r, "q_r", torch.bfloat16, (B, NUM_HEADS, D_R))
    _need(block_table, "block_table", torch.int32)
    _need(o_lat, "o_lat", torch.bfloat16, (B, NUM_HEADS, D_C))
    _need(lse, "lse", torch.float32, (B, NUM_HEADS))
    _need(dev_error, "dev_error", torch.int32, (1,))
    if block_table.dim() != 2 or block_table.shape[0] * max(1, int(info.queries_per_seq)) != B:
        raise ValueError("block_table must be [sequences, max_pages] (query rows / queries_per_seq)")
    dtype = _kv_dtype(kv_pool, kv_scale, kr_pool)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().mla_decode_paged(ctypes.byref(info), _ptr(plan_dev), _ptr(q_abs), _ptr(q_r), dtype, _ptr(kv_pool),
                                _ptr(kv_scale), _ptr(kr_pool), int(kv_pool.shape[0]), _ptr(block_table),
                                int(block_table.shape[1]), float(softmax_scale), _ptr(workspace), ws_bytes,
                                _ptr(o_lat), _ptr(lse), _ptr(dev_error), _stream(stream))
    _check("mla_decode_paged", st)


def mla_absorb_decode_paged(info: PlanInfo, plan_dev: torch.Tensor, q_c: torch.Tensor, w_uk: torch.Tensor,
                            q_abs: torch.Tensor, absorb_sync: torch.Tensor, q_r: torch.Tensor, *,
                            kv_pool: torch.Tensor, block_table: torch.Tensor, o_lat: torch.Tensor, lse: torch.Tensor,
                            dev_error: torch.Tensor, workspace: Optional[torch.Tensor] = None,
                            kv_scale: Optional[torch.Tensor] = None, kr_pool: Optional[torch.Tensor] = None,
                            softmax_scale: float = SOFTMAX_SCALE, stream=None) -> None:
    """Absorb and decode in one launch (the absorb as the decode kernel's prologue); q_abs is
    written.  absorb_sync: int32 [2] on the device, zero before the first call (left zero by
    every call that reports no device error)."""
    B = q_c.shape[0]
    _need(plan_dev, "plan_dev", torch.int32)
    _need(q_c, "q_c", torch.bfloat16, (B, NUM_HEADS, D_HC))
    _need(w_uk, "w_uk", torch.bfloat16, (NUM_HEADS, D_HC, D_C))
    _need(q_abs, "q_abs", torch.bfloat16, (B, NUM_HEADS, D_C))
    _need(absorb_sync, "absorb_sync", torch.int32, (2,))
    _need(q_r, "q_r", torch.bfloat16, (B, NUM_HEADS, D_R))
    _need(block_table, "block_table", torch.int32)
    _need(o_lat, "o_lat", torch.bfloat16, (B, NUM_HEADS, D_C))
    _need(lse, "lse", torch.float32, (B, NUM_HEADS))
    _need(dev_error, "dev_error", torch.int32, (1,))
    if block_table.dim() != 2 or block_table.shape[0] * max(1, int(info.queries_per_seq)) != B:
        raise ValueError("block_table must be [sequences, max_pages] (query rows / queries_per_seq)")
    dtype = _kv_dtype(kv_pool, kv_scale, kr_pool)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().mla_absorb_decode_paged(ctypes.byref(info), _ptr(plan_dev), _ptr(q_c), _ptr(w_uk), _ptr(q_abs),
                                       _ptr(absorb_sync), _ptr(q_r), dtype, _ptr(kv_pool), _ptr(kv_scale),
                                       _ptr(kr_pool), int(kv_pool.shape[0]), _ptr(block_table),
                                       int(block_table.shape[1]), float(softmax_scale), _ptr(workspace), ws_bytes,
                                       _ptr(o_lat), _ptr(lse), _ptr(dev_error), _stream(stream))
    _check("mla_absorb_decode_paged", st)


def mla_decode_paged_static_ws(info: PlanInfo, plan_dev: torch.Tensor, q_abs: torch.Tensor, q_r: torch.Tensor, *,
                               kv_pool: torch.Tensor, block_table: torch.Tensor, o_lat: torch.Tensor,
                               lse: torch.Tensor, dev_error: torch.Tensor, kv_scale: Optional[torch.Tensor] = None,
                               kr_pool: Optional[torch.Tensor] = None, softmax_scale: float = SOFTMAX_SCALE,
                               stream=None) -> None:
    """Decode plus split merge with the library's fixed scratch array: allocates nothing.
    Calls that may overlap on one device race on that array (see include/mla.h)."""
    B = q_abs.shape[0]
    _need(plan_dev, "plan_dev", torch.int32)
    _need(q_abs, "q_abs", torch.bfloat16, (B, NUM_HEADS, D_C))
    _need(q_r, "q_r", torch.bfloat16, (B, NUM_HEADS, D_R))
    _need(block_table, "block_table", torch.int32)
    _need(o_lat, "o_lat", torch.bfloat16, (B, NUM_HEADS, D_C))
    _need(lse, "lse", torch.float32, (B, NUM_HEADS))
    _need(dev_error, "dev_error", torch.int32, (1,))
    if block_table.dim() != 2 or block_table.shape[0] * max(1, int(info.queries_per_seq)) != B:
        raise ValueError("block_table must be [sequences, max_pages] (query rows / queries_per_seq)")
    dtype = _kv_dtype(kv_pool, kv_scale, kr_pool)
    st = lib().mla_decode_paged_static_ws(ctypes.byref(info), _ptr(plan_dev), _ptr(q_abs), _ptr(q_r), dtype,
                                          _ptr(kv_pool), _ptr(kv_scale), _ptr(kr_pool), int(kv_pool.shape[0]),
                                          _ptr(block_table), int(block_table.shape[1]), float(softmax_scale),
                                          _ptr(o_lat), _ptr(lse), _ptr(dev_error), _stream(stream))
    _check("mla_decode_paged_static_ws", st)


def _kv_dtype(kv_pool, kv_scale, kr_pool) -> int:
    if kv_scale is None:
        _need(kv_pool, "kv_pool", torch.bfloat16)
        if kv_pool.dim() != 3 or tuple(kv_pool.shape[1:]) != (PAGE, D_ROW):
            raise ValueError("bf16 kv_pool must be [pages, 64, 576]")
        return MLA_KV_BF16
    _need(kv_pool, "kv_pool (e4m3 codes or NVFP4 rows)", torch.uint8)
    if kv_pool.dim() == 3 and tuple(kv_pool.shape[1:]) == (PAGE, NVFP4_ROW):
        _need(kv_scale, "kv_scale", torch.float32, (kv_pool.shape[0], PAGE))
        _need(kr_pool, "kr_pool", torch.bfloat16, (kv_pool.shape[0], PAGE, D_R))
        return MLA_KV_NVFP4
    if kv_pool.dim() != 3 or tuple(kv_pool.shape[1:]) != (PAGE, D_C):
        raise ValueError("fp8 kv_pool must be [pages, 64, 512] (NVFP4: [pages, 64, 288])")
    _need(kv_scale, "kv_scale", torch.float32, (kv_pool.shape[0], PAGE))
    _need(kr_pool, "kr_pool", torch.bfloat16, (kv_pool.shape[0], PAGE, D_R))
    return MLA_KV_FP8_E4M3


def mla_combine_splits(info: PlanInfo, plan_dev: torch.Tensor, workspace: Optional[torch.Tensor],
                       o_lat: torch.Tensor, lse: torch.Tensor, stream=None) -> None:
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().mla_combine_splits(ctypes.byref(info), _ptr(plan_dev), _ptr(workspace), ws_bytes, _ptr(o_lat),
                                  _ptr(lse), _stream(stream))
    _check("mla_combine_splits", st)


def mla_merge_out_proj(info: PlanInfo, plan_dev: torch.Tensor, workspace: Optional[torch.Tensor],
                       o_lat: torch.Tensor, lse: torch.Tensor, w_uv: torch.Tensor, out: torch.Tensor,
                       dev_error: Optional[torch.Tensor] = None, stream=None) -> None:
    """Split merge and W_UV projection in one launch (merged rows as mla_combine_splits writes
    them, out as mla_out_proj computes it)."""
    B = int(info.batch)
    _need(o_lat, "o_lat", torch.bfloat16, (B, NUM_HEADS, D_C))
    _need(lse, "lse", torch.float32, (B, NUM_HEADS))
    _need(w_uv, "w_uv", torch.bfloat16, (NUM_HEADS, D_HC, D_C))
    _need(out, "out", torch.bfloat16, (B, NUM_HEADS, D_HC))
    if dev_error is not None:
        _need(dev_error, "dev_error", torch.int32, (1,))
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().mla_merge_out_proj(ctypes.byref(info), _ptr(plan_dev), _ptr(workspace), ws_bytes, _ptr(o_lat),
                                  _ptr(lse), _ptr(w_uv), _ptr(out), _ptr(dev_error), _stream(stream))
    _check("mla_merge_out_proj", st)


def mla_append_kv(c_kv: torch.Tensor, k_r: torch.Tensor, slots: torch.Tensor, *, kv_pool: torch.Tensor,
                  dev_error: torch.Tensor, kv_scale: Optional[torch.Tensor] = None,
                  kr_pool: Optional[torch.Tensor] = None, stream=None) -> None:
    """Write new tokens into the paged cache: token i to slot slots[i] (page * 64 + row; negative
    = skip).  bf16 cache: kv_pool [pages, 64, 576].  FP8 cache (kv_scale given): c_KV quantised
    per token into kv_pool [pages, 64, 512] (e4m3 codes) and kv_scale [pages, 64], k_R into
    kr_pool [pages, 64, 64]."""
    if not isinstance(slots, torch.Tensor) or slots.dim() != 1:
        raise ValueError("slots must be a 1-d tensor")
    n = int(slots.shape[0])
    _need(slots, "slots", torch.int32, (n,))
    _need(c_kv, "c_kv", torch.bfloat16, (n, D_C))
    _need(k_r, "k_r", torch.bfloat16, (n, D_R))
    _need(dev_error, "dev_error", torch.int32, (1,))
    dtype = _kv_dtype(kv_pool, kv_scale, kr_pool)
    st = lib().mla_append_kv(n, _ptr(c_kv), _ptr(k_r), _ptr(slots), dtype, int(kv_pool.shape[0]), _ptr(kv_pool),
                             _ptr(kv_scale), _ptr(kr_pool), _ptr(dev_error), _stream(stream))
    _check("mla_append_kv", st)


def mla_gather_kv(*, kv_pool: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                  cu_seqlens: torch.Tensor, out: torch.Tensor, dev_error: torch.Tensor,
                  kv_scale: Optional[torch.Tensor] = None, kr_pool: Optional[torch.Tensor] = None,
                  stream=None) -> None:
    """Every sequence's cache rows in logical order into out [total, 576] (bf16), dequantised
    from an FP8 or NVFP4 cache; cu_seqlens [B + 1] gives each sequence's first row."""
    dtype = _kv_dtype(kv_pool, kv_scale, kr_pool)
    _need(block_table, "block_table", torch.int32)
    B = int(seq_lens.shape[0])
    _need(seq_lens, "seq_lens", torch.int32, (B,))
    _need(cu_seqlens, "cu_seqlens", torch.int32, (B + 1,))
    _need(out, "out", torch.bfloat16)
    _need(dev_error, "dev_error", torch.int32, (1,))
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [batch, max_pages]")
    if out.dim() != 2 or out.shape[1] != D_ROW:
        raise ValueError("out must be [total tokens, 576]")
    st = lib().mla_gather_kv(dtype, _ptr(kv_pool), _ptr(kv_scale), _ptr(kr_pool), int(kv_pool.shape[0]),
                             _ptr(block_table), int(block_table.shape[1]), _ptr(seq_lens), _ptr(cu_seqlens), B,
                             _ptr(out), _ptr(dev_error), _stream(stream))
    _check("mla_gather_kv", st)


# --------------------------------------------------------------------------- rotary positions

class Rope:
    """The constants of a rotation (``mla_rope_config``), made once: ``dim`` rotated elements per
    head, ``layout`` "interleaved" (pairs 2i, 2i + 1) or "half" (pairs i, i + dim / 2), frequencies
    base^(-2i / dim) with ``scaling`` "none", "linear" (divided by ``factor``) or "yarn" (``factor``
    over ``original_len`` trained positions), or the caller's ``inv_freq`` [dim / 2] as they are.
    ``magnitude`` multiplies cos and sin (0: the scaling's own, for "yarn" m = 0.1 ln(factor) + 1,
    which is the attention temperature of a head that is rotated as a whole).  For DecodeStep, whose
    heads are rotated in 64 of 192 elements, YaRN is magnitude=1.0 here and softmax_scale = m^2 /
    sqrt(192) there."""

    def __init__(self, dim: int = D_R, *, base: float = 10000.0, layout: str = "interleaved", scaling: str = "none",
                 factor: float = 1.0, original_len: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0,
                 magnitude: float = 0.0, inv_freq=None):
        if layout not in _ROPE_LAYOUTS:
            raise ValueError(f"layout must be one of {tuple(_ROPE_LAYOUTS)}, got {layout!r}")
        if scaling not in _ROPE_SCALINGS:
            raise ValueError(f"scaling must be one of {tuple(_ROPE_SCALINGS)}, got {scaling!r}")
        freq = None
        if inv_freq is not None:
            freq = np.ascontiguousarray(np.asarray(inv_freq, dtype=np.float64))
            if freq.shape != (int(dim) // 2,):
                raise ValueError("inv_freq must hold dim / 2 frequencies")
        opts = RopeOptions(int(dim), _ROPE_LAYOUTS[layout], _ROPE_SCALINGS[scaling], int(original_len), float(base),
                           float(factor), float(beta_fast), float(beta_slow), float(magnitude),
                           None if freq is None else freq.ctypes.data)
        self.config = RopeConfig()
        _check("mla_rope_init", lib().mla_rope_init(ctypes.byref(opts), ctypes.byref(self.config)))
        self.dim, self.layout, self.magnitude = int(dim), layout, float(self.config.magnitude)
        self._ref = ctypes.byref(self.config)


def _refuse(t, name: str, dtype, shape, device: int):
    """The error of a tensor that failed one of its checks."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name}: expected shape {shape}, got {tuple(t.shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name}: must be on the current CUDA device ({device}), is on {t.device}")
    raise ValueError(f"{name}: must be contiguous (rows of a wider tensor: in the last dimension)")


def _rows(t, name: str, dtype, shape, device: int) -> int:
    """The address of a tensor of that type and shape on the current device (where the kernel is
    launched); any strides but the last, which is 1."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or t.get_device() != device or \
            (t.stride(-1) != 1 and shape[-1] > 1):
        _refuse(t, name, dtype, shape, device)
    return t.data_ptr()


def _whole(t, name: str, dtype, shape, device: int) -> int:
    """The address of a contiguous tensor of that type and shape on the current device."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or t.get_device() != device or \
            not t.is_contiguous():
        _refuse(t, name, dtype, shape, device)
    return t.data_ptr()


def mla_rope(rope: Rope, x: torch.Tensor, positions: torch.Tensor, out: Optional[torch.Tensor] = None, *,
             rest: Optional[torch.Tensor] = None, rot_offset: int = 0, stream=None) -> torch.Tensor:
    """Rotate elements [rot_offset, rot_offset + rope.dim) of every head of x [tokens, heads,
    head_dim] (bf16, fp16 or fp32; any strides, the last 1) by positions (int32 [tokens]) into
    out, which it returns: x itself (None: in place), a tensor like x (the other elements copied),
    or, with ``rest`` [tokens, heads, head_dim - dim], one of [tokens, heads, dim]."""
    device = torch._C._cuda_getDevice()
    if out is None and rest is None:
        out = x
    try:  # the checks in one expression; what it refuses is told by _check_rope
        dtype, dim, (T, H, D), (xt, xh, xd), (ot, oh, od) = x.dtype, rope.dim, x.shape, x.stride(), out.stride()
        code = _DTYPES.get(dtype)
        rest_ptr, rt, rh = None, 0, 0
        fine = code is not None and xd == 1 and od == 1 and out.dtype is dtype and x.get_device() == device and \
            out.get_device() == device and positions.dtype is torch.int32 and positions.shape == (T,) and \
            positions.get_device() == device and positions.is_contiguous()
        if rest is None:
            fine = fine and out.shape == x.shape
        else:
            rt, rh, rd = rest.stride()
            rest_ptr = rest.data_ptr()
            fine = fine and (rd == 1 or D - dim == 1) and rest.dtype is dtype and rest.get_device() == device and \
                out.shape == (T, H, dim) and rest.shape == (T, H, D - dim)
    except (AttributeError, TypeError, ValueError):
        fine = False
    if not fine:
        _check_rope(rope, x, positions, out, rest, device)
    st = lib().mla_rope(rope._ref, code, T, H, D, rot_offset, x.data_ptr(), xt, xh, out.data_ptr(), ot, oh, rest_ptr, rt,
                        rh, positions.data_ptr(), _stream(stream))
    if st:
        _check("mla_rope", st)
    return out


def _check_rope(rope, x, positions, out, rest, device: int) -> None:
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("x must be [tokens, heads, head_dim]")
    if x.dtype not in _DTYPES:
        raise TypeError(f"x: expected bfloat16, float16 or float32, got {x.dtype}")
    T, H, D = x.shape
    if out is None:
        raise ValueError("rest needs out")
    _rows(x, "x", x.dtype, (T, H, D), device)
    _rows(out, "out", x.dtype, (T, H, D if rest is None else rope.dim), device)
    if rest is not None:
        _rows(rest, "rest", x.dtype, (T, H, D - rope.dim), device)
    _whole(positions, "positions", torch.int32, (T,), device)
    raise ValueError("mla_rope: arguments that do not fit together")


def mla_rope_append_kv(rope: Rope, c_kv: torch.Tensor, k_r: torch.Tensor, positions: torch.Tensor,
                       slots: torch.Tensor, *, kv_pool: torch.Tensor, dev_error: torch.Tensor,
                       kv_scale: Optional[torch.Tensor] = None, kr_pool: Optional[torch.Tensor] = None,
                       q: Optional[torch.Tensor] = None, q_c: Optional[torch.Tensor] = None,
                       q_r: Optional[torch.Tensor] = None, stream=None) -> None:
    """mla_append_kv with k_r rotated by the tokens' positions on the way; c_kv [n, 512] and k_r
    [n, 64] may be columns of a wider row.  With q [n, 128, 192] (content, then un-rotated part;
    any strides, the last 1), q_c [n, 128, 128] and q_r [n, 128, 64] receive the split and rotated
    queries in the same launch."""
    bf16, i32, device = torch.bfloat16, torch.int32, torch._C._cuda_getDevice()
    scale_ptr = kr_ptr = q_ptr = qc_ptr = qr_ptr = None
    qt = qh = 0
    try:  # the checks in one expression; what it refuses is told by _check_rope_append
        n, (pages, _, width) = slots.numel(), kv_pool.shape
        (cs, c1), (ks, k1) = c_kv.stride(), k_r.stride()
        fine = slots.dtype is i32 and slots.shape == (n,) and slots.is_contiguous() and slots.get_device() == device and \
            positions.dtype is i32 and positions.shape == (n,) and positions.is_contiguous() and \
            positions.get_device() == device and c_kv.dtype is bf16 and c_kv.shape == (n, D_C) and c1 == 1 and \
            c_kv.get_device() == device and k_r.dtype is bf16 and k_r.shape == (n, D_R) and k1 == 1 and \
            k_r.get_device() == device and dev_error.dtype is i32 and dev_error.shape == (1,) and \
            dev_error.get_device() == device and kv_pool.is_contiguous() and kv_pool.get_device() == device and \
            kv_pool.shape[1] == PAGE
        if kv_scale is None:
            dtype = MLA_KV_BF16
            fine = fine and kv_pool.dtype is bf16 and width == D_ROW
        else:
            dtype = MLA_KV_NVFP4 if width == NVFP4_ROW else MLA_KV_FP8_E4M3
            fine = fine and kv_pool.dtype is torch.uint8 and (width == D_C or width == NVFP4_ROW) and \
                kv_scale.dtype is torch.float32 and kv_scale.shape == (pages, PAGE) and kv_scale.is_contiguous() and \
                kv_scale.get_device() == device and kr_pool.dtype is bf16 and kr_pool.shape == (pages, PAGE, D_R) and \
                kr_pool.is_contiguous() and kr_pool.get_device() == device
            scale_ptr, kr_ptr = kv_scale.data_ptr(), kr_pool.data_ptr()
        if q is not None:
            qt, qh, q1 = q.stride()
            fine = fine and q.dtype is bf16 and q.shape == (n, NUM_HEADS, D_HC + D_R) and q1 == 1 and \
                q.get_device() == device and q_c.dtype is bf16 and q_c.shape == (n, NUM_HEADS, D_HC) and \
                q_c.is_contiguous() and q_c.get_device() == device and q_r.dtype is bf16 and \
                q_r.shape == (n, NUM_HEADS, D_R) and q_r.is_contiguous() and q_r.get_device() == device
            q_ptr, qc_ptr, qr_ptr = q.data_ptr(), q_c.data_ptr(), q_r.data_ptr()
        else:
            fine = fine and q_c is None and q_r is None
    except (AttributeError, TypeError, ValueError):
        fine = False
    if not fine:
        _check_rope_append(c_kv, k_r, positions, slots, kv_pool, dev_error, kv_scale, kr_pool, q, q_c, q_r, device)
    st = lib().mla_rope_append_kv(rope._ref, n, c_kv.data_ptr(), cs, k_r.data_ptr(), ks, positions.data_ptr(),
                                  slots.data_ptr(), dtype, pages, kv_pool.data_ptr(), scale_ptr, kr_ptr, q_ptr, qt, qh,
                                  qc_ptr, qr_ptr, dev_error.data_ptr(), _stream(stream))
    if st:
        _check("mla_rope_append_kv", st)


def _check_rope_append(c_kv, k_r, positions, slots, kv_pool, dev_error, kv_scale, kr_pool, q, q_c, q_r,
                       device: int) -> None:
    if not isinstance(slots, torch.Tensor) or slots.dim() != 1:
        raise ValueError("slots must be a 1-d tensor")
    n, bf16, i32 = slots.shape[0], torch.bfloat16, torch.int32
    _whole(slots, "slots", i32, (n,), device)
    _whole(positions, "positions", i32, (n,), device)
    _rows(c_kv, "c_kv", bf16, (n, D_C), device)
    _rows(k_r, "k_r", bf16, (n, D_R), device)
    _whole(dev_error, "dev_error", i32, (1,), device)
    _kv_dtype(kv_pool, kv_scale, kr_pool)
    for name, t in (("kv_pool", kv_pool), ("kv_scale", kv_scale), ("kr_pool", kr_pool)):
        if t is not None:
            _whole(t, name, t.dtype, tuple(t.shape), device)
    if q is not None:
        _rows(q, "q", bf16, (n, NUM_HEADS, D_HC + D_R), device)
        _whole(q_c, "q_c", bf16, (n, NUM_HEADS, D_HC), device)
        _whole(q_r, "q_r", bf16, (n, NUM_HEADS, D_R), device)
    elif q_c is not None or q_r is not None:
        raise ValueError("q_c and q_r need q")
    raise ValueError("mla_rope_append_kv: arguments that do not fit together")


# --------------------------------------------------------------------------- 4-bit weights

class W4Weight:
    """Weights [heads, n, k] in 4 bits, laid out once for the products (``mla_w4_pack``, on the current
    stream; the tensors given are not kept): ``codes`` uint8 [heads, n, k / 2] (value 2j in the low
    nibble of byte j) and a ``scale`` per group of k.  A bfloat16 scale [heads, n, k / group], group
    32, 64 or 128: int4, (code - zero) * scale, ``zero`` uint8 of the scale's shape (None: 8).  A
    uint8 or float8_e4m3fn scale [heads, n, k / 16]: NVFP4, e2m1(code) * e4m3(scale).
    ``tensor_scale`` multiplies every output.  Tensors without the leading dimension are one head.
    For the decode step: W_UK as [128, 512, 128] (c, then d) and W_UV as [128, 128, 512]."""

    def __init__(self, codes: torch.Tensor, scale: torch.Tensor, *, zero: Optional[torch.Tensor] = None,
                 group: Optional[int] = None, tensor_scale: float = 1.0):
        for name, t in (("codes", codes), ("scale", scale)) + ((("zero", zero),) if zero is not None else ()):
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{name}: expected a tensor")
            if t.dim() not in (2, 3) or t.dim() != codes.dim():
                raise ValueError(f"{name}: must be [heads, n, ...] or [n, ...] like codes")
        if scale.dtype == torch.float8_e4m3fn:
            scale = scale.view(torch.uint8)
        if scale.dtype not in (torch.bfloat16, torch.uint8):
            raise TypeError(f"scale: expected bfloat16 (int4), uint8 or float8_e4m3fn (NVFP4), got {scale.dtype}")
        self.format = MLA_W4_INT4 if scale.dtype == torch.bfloat16 else MLA_W4_NVFP4
        heads, n = (1, codes.shape[0]) if codes.dim() == 2 else codes.shape[:2]
        k = 2 * codes.shape[-1]
        groups = scale.shape[-1]
        if groups < 1 or k % groups or (group is not None and k != groups * group):
            raise ValueError(f"scale: {groups} groups do not divide k = {k}" +
                             ("" if group is None else f" into groups of {group}"))
        self.heads, self.n, self.k, self.group = int(heads), int(n), int(k), k // groups
        self.tensor_scale = float(tensor_scale)
        allowed = (32, 64, 128) if self.format == MLA_W4_INT4 else (16,)
        if self.group not in allowed or k % 32:
            raise ValueError(f"groups of {self.group} over k = {k}: expected groups of {allowed} and k a multiple of 32")
        if zero is not None and self.format == MLA_W4_NVFP4:
            raise ValueError("zero points are for int4")
        device = torch._C._cuda_getDevice()
        codes_ptr = _whole(codes, "codes", torch.uint8, tuple(codes.shape), device)
        scale_ptr = _whole(scale, "scale", scale.dtype, tuple(codes.shape[:-1]) + (groups,), device)
        zero_ptr = None if zero is None else _whole(zero, "zero", torch.uint8, tuple(scale.shape), device)
        self.device_index = device
        self.struct = W4Struct(self.format, self.heads, self.n, self.k, self.group, int(zero is not None),
                               self.tensor_scale, None)
        self._ref = ctypes.byref(self.struct)
        size = int(lib().mla_w4_packed_bytes(self._ref))
        if size == 0:
            raise MlaError("mla_w4_packed_bytes", MLA_ERR_UNSUPPORTED, "sizes past the limits")
        self.packed = torch.empty(size, dtype=torch.uint8, device=codes.device)
        _check("mla_w4_pack", lib().mla_w4_pack(self._ref, codes_ptr, scale_ptr, zero_ptr, self.packed.data_ptr(),
                                                _stream(None)))
        self.struct.packed = self.packed.data_ptr()


def mla_linear_w4(x: torch.Tensor, w: W4Weight, out: torch.Tensor, stream=None) -> None:
    """out[r, h, :] = W[h] x[r, h, :] for the few rows of a decode batch: x [rows, heads, k] and out
    [rows, heads, n] bf16 (heads 1: [rows, k] and [rows, n] too), any strides, the last 1; x may be
    expanded over the heads."""
    if not isinstance(x, torch.Tensor) or not isinstance(out, torch.Tensor):
        raise TypeError("x and out: expected tensors")
    heads, device = w.heads, torch._C._cuda_getDevice()
    if heads == 1:
        x = x.unsqueeze(1) if x.dim() == 2 else x
        out = out.unsqueeze(1) if out.dim() == 2 else out
    rows, bf16 = x.shape[0], torch.bfloat16
    x_ptr = _rows(x, "x", bf16, (rows, heads, w.k), device)
    out_ptr = _rows(out, "out", bf16, (rows, heads, w.n), device)
    if w.device_index != device:
        raise ValueError(f"w: must be on the current CUDA device ({device})")
    (xr, xh, _), (o_r, oh, _) = x.stride(), out.stride()
    st = lib().mla_linear_w4(rows, x_ptr, xr, xh, w._ref, out_ptr, o_r, oh, _stream(stream))
    if st:
        _check("mla_linear_w4", st)


def _head_product(fn: str, x: torch.Tensor, w: W4Weight, out: torch.Tensor, names, k: int, n: int, stream) -> None:
    B, device = x.shape[0], torch._C._cuda_getDevice()
    x_ptr = _whole(x, names[0], torch.bfloat16, (B, NUM_HEADS, k), device)
    out_ptr = _whole(out, names[1], torch.bfloat16, (B, NUM_HEADS, n), device)
    if (w.heads, w.n, w.k) != (NUM_HEADS, n, k):
        raise ValueError(f"weights: expected [{NUM_HEADS}, {n}, {k}], got [{w.heads}, {w.n}, {w.k}]")
    if w.device_index != device:
        raise ValueError(f"weights: must be on the current CUDA device ({device})")
    st = getattr(lib(), fn)(x_ptr, w._ref, out_ptr, B, _stream(stream))
    if st:
        _check(fn, st)


def mla_absorb_q_w4(q_c: torch.Tensor, w_uk: W4Weight, q_abs: torch.Tensor, stream=None) -> None:
    """mla_absorb_q with W_UK in 4 bits, laid out [128, 512, 128] (groups along d_hc)."""
    _head_product("mla_absorb_q_w4", q_c, w_uk, q_abs, ("q_c", "q_abs"), D_HC, D_C, stream)


def mla_out_proj_w4(o_lat: torch.Tensor, w_uv: W4Weight, out: torch.Tensor, stream=None) -> None:
    """mla_out_proj with W_UV in 4 bits, laid out [128, 128, 512] (groups along d_c)."""
    _head_product("mla_out_proj_w4", o_lat, w_uv, out, ("o_lat", "out"), D_C, D_HC, stream)


# Chunks of at least this many new tokens take the decompressed form, shorter ones the absorbed
# decode (page 1 section 3, kPrefillThresh in mla_config.h; section 6 measures the switch).  Under a
# window the decompression is of the window alone and pays much earlier: from some 16 new tokens on under
# 512, 32 to 64 under 1,024, 64 to 96 under 4,096 (255 tokens under 1,024: some 155 us absorbed, 71 in the
# chunk form).  The default is the same there, and `threshold` says otherwise.
PREFILL_THRESHOLD = 256


def mla_prefill_decompressed(*, kv_pool: torch.Tensor, block_table_row: torch.Tensor, seq_len: int,
                             q_c: torch.Tensor, q_r: torch.Tensor, w_uk: torch.Tensor, w_uv: torch.Tensor,
                             out: torch.Tensor, dev_error: torch.Tensor, workspace: Optional[torch.Tensor] = None,
                             kv_scale: Optional[torch.Tensor] = None, kr_pool: Optional[torch.Tensor] = None,
                             softmax_scale: float = SOFTMAX_SCALE, stream=None) -> None:
    """The last T = q_c.shape[0] tokens of one sequence of seq_len cached tokens, attended
    causally in the decompressed form: out [T, 128, 128].  workspace: at least
    mla_prefill_workspace_bytes(seq_len) bytes (allocated here when None)."""
    T = int(q_c.shape[0])
    _need(q_c, "q_c", torch.bfloat16, (T, NUM_HEADS, D_HC))
    _need(q_r, "q_r", torch.bfloat16, (T, NUM_HEADS, D_R))
    _need(out, "out", torch.bfloat16, (T, NUM_HEADS, D_HC))
    _need(block_table_row, "block_table_row", torch.int32)
    _need(dev_error, "dev_error", torch.int32, (1,))
    need = int(lib().mla_prefill_workspace_bytes(int(seq_len)))
    if workspace is None:
        workspace = _scratch(need, q_c.device, stream)
    ws_bytes = workspace.numel() * workspace.element_size()
    dtype = _kv_dtype(kv_pool, kv_scale, kr_pool)
    st = lib().mla_prefill_decompressed(dtype, _ptr(kv_pool), _ptr(kv_scale), _ptr(kr_pool), int(kv_pool.shape[0]),
                                        _ptr(block_table_row), int(block_table_row.numel()), int(seq_len), T,
                                        _ptr(q_c), _ptr(q_r), _ptr(w_uk), _ptr(w_uv), float(softmax_scale),
                                        _ptr(workspace), ws_bytes, _ptr(out), _ptr(dev_error), _stream(stream))
    _check("mla_prefill_decompressed", st)


def prefill_chunk(seq_len: int, q_c: torch.Tensor, q_r: torch.Tensor, *, w_uk: torch.Tensor, w_uv: torch.Tensor,
                  kv_pool: torch.Tensor, block_table_row: torch.Tensor, kv_scale: Optional[torch.Tensor] = None,
                  kr_pool: Optional[torch.Tensor] = None, threshold: int = PREFILL_THRESHOLD,
                  softmax_scale: float = SOFTMAX_SCALE, window: int = 0, sinks: int = 0, stream=None):
    """A chunk of T = q_c.shape[0] new tokens at the end of one sequence of seq_len cached
    tokens (the chunk's cache rows included): chunks shorter than `threshold` run the absorbed
    decode with T query rows (DecodeStep, queries_per_seq = T), longer ones the decompressed
    form (mla_prefill_decompressed; with a ``window`` mla_prefill_window).  Returns
    (out [T, 128, 128], device error word)."""
    T = int(q_c.shape[0])
    bt = block_table_row.reshape(1, -1)
    with _on(stream, q_c.device):  # the plan, the buffers and their zeros too
        if T < threshold:
            step = DecodeStep(np.array([seq_len], np.int32), w_uk=w_uk, w_uv=w_uv, kv_pool=kv_pool, block_table=bt,
                              kv_scale=kv_scale, kr_pool=kr_pool, device=q_c.device, queries_per_seq=T,
                              softmax_scale=softmax_scale, window=window, sinks=sinks)
            return step.run(q_c, q_r), step.dev_error
        if isinstance(w_uk, W4Weight) or isinstance(w_uv, W4Weight):
            raise ValueError(f"prefill_chunk: chunks of {threshold} or more new tokens read bf16 weights")
        if sinks and not window:
            raise ValueError("sinks need a window")
        out = torch.empty(T, NUM_HEADS, D_HC, dtype=torch.bfloat16, device=q_c.device)
        err = torch.zeros(1, dtype=torch.int32, device=q_c.device)
        attend = partial(mla_prefill_window, window=window, sinks=sinks) if window else mla_prefill_decompressed
        attend(kv_pool=kv_pool, block_table_row=bt[0], seq_len=seq_len, q_c=q_c, q_r=q_r, w_uk=w_uk, w_uv=w_uv, out=out,
               dev_error=err, kv_scale=kv_scale, kr_pool=kr_pool, softmax_scale=softmax_scale)
        return out, err


# --------------------------------------------------------------------------- windows and shared prefixes

def mla_prefill_window_workspace_bytes(seq_len: int, chunk_len: int, window: int, sinks: int = 0) -> int:
    size = int(lib().mla_prefill_window_workspace_bytes(_i32(seq_len), _i32(chunk_len), _i32(window), _i32(sinks)))
    if size == 0:
        raise MlaError("mla_prefill_window_workspace_bytes", MLA_ERR_INVALID_ARG, "invalid sizes")
    return size


def mla_prefill_window(*, kv_pool: torch.Tensor, block_table_row: torch.Tensor, seq_len: int, window: int,
                       q_c: torch.Tensor, q_r: torch.Tensor, w_uk: torch.Tensor, w_uv: torch.Tensor, out: torch.Tensor,
                       dev_error: torch.Tensor, sinks: int = 0, workspace: Optional[torch.Tensor] = None,
                       kv_scale: Optional[torch.Tensor] = None, kr_pool: Optional[torch.Tensor] = None,
                       softmax_scale: float = SOFTMAX_SCALE, stream=None) -> None:
    """mla_prefill_decompressed under a sliding window: the query at position p sees the last
    ``window`` positions up to its own and the first ``sinks``.  workspace: a uint8 tensor of at least
    mla_prefill_window_workspace_bytes(seq_len, chunk, window, sinks) (allocated here when None)."""
    device = torch._C._cuda_getDevice()
    if not isinstance(q_c, torch.Tensor) or q_c.dim() != 3:
        raise ValueError("q_c must be [chunk, 128, 128]")
    T, bf16 = int(q_c.shape[0]), torch.bfloat16
    ptrs = [_whole(t, name, bf16, shape, device) for t, name, shape in (
        (q_c, "q_c", (T, NUM_HEADS, D_HC)), (q_r, "q_r", (T, NUM_HEADS, D_R)), (w_uk, "w_uk", (NUM_HEADS, D_HC, D_C)),
        (w_uv, "w_uv", (NUM_HEADS, D_HC, D_C)))]
    out_ptr = _whole(out, "out", bf16, (T, NUM_HEADS, D_HC), device)
    cache = _cache(kv_pool, kv_scale, kr_pool, device)
    table, pages = _table_row(block_table_row, device)
    err = _whole(dev_error, "dev_error", torch.int32, (1,), device)
    if workspace is None:
        workspace = _scratch(mla_prefill_window_workspace_bytes(seq_len, T, window, sinks), q_c.device, stream)
    ws = _whole(workspace, "workspace", workspace.dtype, tuple(workspace.shape), device)
    st = lib().mla_prefill_window(*cache, table, pages, _i32(seq_len), T, _i32(window), _i32(sinks), *ptrs,
                                  float(softmax_scale), ws, workspace.numel() * workspace.element_size(), out_ptr, err,
                                  _stream(stream))
    if st:
        _check("mla_prefill_window", st)


def _on(stream, device):
    """A context with the stream that a call is sent to as the current one: what is allocated or filled in it
    is that stream's, so that what is let go of when the call returns is handed out again on that stream
    alone, behind the call's kernels."""
    if stream is not None:
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        if handle != _stream(None):
            # (an ExternalStream of 0 would be a new stream, not the default one)
            return torch.cuda.stream(torch.cuda.ExternalStream(handle, device=device) if handle else
                                     torch.cuda.default_stream(device))
    return nullcontext()


def _scratch(size: int, device, stream) -> torch.Tensor:
    """A workspace of one call on ``stream``, from that stream's memory."""
    with _on(stream, device):
        return torch.empty(max(16, size), dtype=torch.uint8, device=device)


def _cache(kv_pool, kv_scale, kr_pool, device: int):
    """The leading arguments of a call that reads a cache of any of the three kinds."""
    try:  # the checks in one expression; what it refuses is told below
        pages, rows, width = kv_pool.shape
        if kv_scale is None:
            dtype, scale_ptr, kr_ptr = MLA_KV_BF16, None, None
            fine = kv_pool.dtype is torch.bfloat16 and width == D_ROW
        else:
            dtype = MLA_KV_NVFP4 if width == NVFP4_ROW else MLA_KV_FP8_E4M3
            fine = kv_pool.dtype is torch.uint8 and (width == D_C or width == NVFP4_ROW) and \
                kv_scale.dtype is torch.float32 and kv_scale.shape == (pages, PAGE) and kv_scale.is_contiguous() and \
                kv_scale.get_device() == device and kr_pool.dtype is torch.bfloat16 and \
                kr_pool.shape == (pages, PAGE, D_R) and kr_pool.is_contiguous() and kr_pool.get_device() == device
            scale_ptr, kr_ptr = kv_scale.data_ptr(), kr_pool.data_ptr()
        fine = fine and rows == PAGE and kv_pool.is_contiguous() and kv_pool.get_device() == device
    except (AttributeError, TypeError, ValueError):
        fine = False
    if not fine:
        _kv_dtype(kv_pool, kv_scale, kr_pool)
        for name, t in (("kv_pool", kv_pool), ("kv_scale", kv_scale), ("kr_pool", kr_pool)):
            if t is not None:
                _whole(t, name, t.dtype, tuple(t.shape), device)
        raise ValueError("cache: arguments that do not fit together")
    return dtype, kv_pool.data_ptr(), scale_ptr, kr_ptr, pages


def _table_row(row, device: int):
    if not isinstance(row, torch.Tensor) or row.dim() != 1:
        raise ValueError("block_table_row must be a 1-d tensor")
    return _whole(row, "block_table_row", torch.int32, tuple(row.shape), device), int(row.shape[0])


class SharedPrefix:
    """A prefix that the sequences of a batch share, decompressed once (``mla_prefix_open``, on the
    current stream) and kept: keys ``k`` and values ``v`` [128 heads, tokens, 128] and rotary keys
    ``k_r`` [tokens, 64], 66.7 KB for each token.  ``block_table_row`` lists the prefix's pages, whose
    last may be partly filled.  For mla_prefix_attend, and for DecodeStep(prefix=...), whose sequences
    are then the tokens behind the prefix.  Faster than block tables that list the shared pages
    themselves from about 48 query rows on with 8,192 shared tokens or more, from about 100 with 2,048."""

    def __init__(self, prefix_len: int, *, w_uk: torch.Tensor, w_uv: torch.Tensor, kv_pool: torch.Tensor,
                 block_table_row: torch.Tensor, kv_scale: Optional[torch.Tensor] = None,
                 kr_pool: Optional[torch.Tensor] = None, dev_error: Optional[torch.Tensor] = None):
        device, bf16, P = torch._C._cuda_getDevice(), torch.bfloat16, int(prefix_len)
        if P < 1:
            raise ValueError(f"prefix_len: expected at least one token, got {P}")
        weights = [_whole(t, name, bf16, (NUM_HEADS, D_HC, D_C), device) for t, name in ((w_uk, "w_uk"), (w_uv, "w_uv"))]
        cache = _cache(kv_pool, kv_scale, kr_pool, device)
        table, pages = _table_row(block_table_row, device)
        where = kv_pool.device
        err = torch.zeros(1, dtype=torch.int32, device=where) if dev_error is None else dev_error
        err_ptr = _whole(err, "dev_error", torch.int32, (1,), device)
        if (P + PAGE - 1) // PAGE > pages:
            raise ValueError(f"block_table_row holds {pages} pages, the prefix needs {(P + PAGE - 1) // PAGE}")
        rows = torch.empty((P, D_ROW), dtype=bf16, device=where)
        k = torch.empty((NUM_HEADS, P, D_HC), dtype=bf16, device=where)
        v = torch.empty((NUM_HEADS, P, D_HC), dtype=bf16, device=where)
        st = lib().mla_prefix_open(*cache, table, pages, P, *weights, rows.data_ptr(), k.data_ptr(), v.data_ptr(), err_ptr,
                                   _stream(None))
        if st:
            _check("mla_prefix_open", st)
        self._set(k, v, rows.narrow(1, D_C, D_R), err, device)

    @classmethod
    def of(cls, k: torch.Tensor, v: torch.Tensor, k_r: torch.Tensor, dev_error: Optional[torch.Tensor] = None):
        """The prefix of keys and values that are there already (bf16; k_r's rows may be columns of wider
        ones, in steps of 8).  The tensors are kept, not copied."""
        device = torch._C._cuda_getDevice()
        P = int(k.shape[1]) if isinstance(k, torch.Tensor) and k.dim() == 3 else 0
        if P < 1:
            raise ValueError("k must be [128, tokens, 128] with at least one token")
        for name, t in (("k", k), ("v", v)):
            _whole(t, name, torch.bfloat16, (NUM_HEADS, P, D_HC), device)
        _rows(k_r, "k_r", torch.bfloat16, (P, D_R), device)
        self = cls.__new__(cls)
        self._set(k, v, k_r, torch.zeros(1, dtype=torch.int32, device=k.device) if dev_error is None else dev_error, device)
        return self

    def _set(self, k, v, k_r, err, device: int) -> None:
        self.k, self.v, self.k_r, self.dev_error, self.device_index = k, v, k_r, err, device
        self.prefix_len = int(k.shape[1])
        self._num_sms = num_sms(device)
        # one token: any stride is that token's
        stride = int(k_r.stride(0)) if self.prefix_len > 1 else D_R
        self._args = (self.prefix_len, self._num_sms), (k.data_ptr(), v.data_ptr(), k_r.data_ptr(), stride)

    def workspace_bytes(self, rows: int) -> int:
        return int(lib().mla_prefix_attend_workspace_bytes(_i32(rows), self.prefix_len, self._num_sms))

    def workspace(self, rows: int) -> torch.Tensor:
        """A workspace for mla_prefix_attend with that many query rows."""
        return torch.empty(max(16, self.workspace_bytes(rows)), dtype=torch.uint8, device=self.k.device)


def mla_prefix_attend(prefix: SharedPrefix, q_c: torch.Tensor, q_r: torch.Tensor, out: torch.Tensor, *,
                      lse: Optional[torch.Tensor] = None, own_out: Optional[torch.Tensor] = None,
                      own_lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                      dev_error: Optional[torch.Tensor] = None, softmax_scale: float = SOFTMAX_SCALE,
                      stream=None) -> None:
    """Attention of all query rows q_c [rows, 128, 128], q_r [rows, 128, 64] to the prefix, merged with
    their attention over their own tokens (own_out [rows, 128, 128] and own_lse [rows, 128]; None: the
    prefix alone) into out and lse, which may be own_out and own_lse themselves.  workspace: a tensor of
    prefix.workspace_bytes(rows) bytes (allocated here when None)."""
    device, bf16 = torch._C._cuda_getDevice(), torch.bfloat16
    if not isinstance(q_c, torch.Tensor) or q_c.dim() != 3:
        raise ValueError("q_c must be [rows, 128, 128]")
    R = int(q_c.shape[0])
    q_c_ptr = _whole(q_c, "q_c", bf16, (R, NUM_HEADS, D_HC), device)
    q_r_ptr = _whole(q_r, "q_r", bf16, (R, NUM_HEADS, D_R), device)
    out_ptr = _whole(out, "out", bf16, (R, NUM_HEADS, D_HC), device)
    lse_ptr = None if lse is None else _whole(lse, "lse", torch.float32, (R, NUM_HEADS), device)
    if (own_out is None) != (own_lse is None):
        raise ValueError("own_out and own_lse: both or neither")
    own_ptr = own_lse_ptr = None
    if own_out is not None:
        own_ptr = _whole(own_out, "own_out", bf16, (R, NUM_HEADS, D_HC), device)
        own_lse_ptr = _whole(own_lse, "own_lse", torch.float32, (R, NUM_HEADS), device)
    if prefix.device_index != device:
        raise ValueError(f"prefix: must be on the current CUDA device ({device})")
    if workspace is None:
        workspace = _scratch(prefix.workspace_bytes(R), q_c.device, stream)
    ws = _whole(workspace, "workspace", workspace.dtype, tuple(workspace.shape), device)
    err = prefix.dev_error if dev_error is None else dev_error
    sizes, keys = prefix._args
    st = lib().mla_prefix_attend(R, *sizes, q_c_ptr, q_r_ptr, *keys, softmax_scale, own_ptr, own_lse_ptr, ws,
                                 workspace.numel() * workspace.element_size(), out_ptr, lse_ptr,
                                 _whole(err, "dev_error", torch.int32, (1,), device), _stream(stream))
    if st:
        _check("mla_prefix_attend", st)


def mla_read_device_error(dev_error: torch.Tensor, stream=None) -> int:
    """Device error bits (0 = none); waits for the stream."""
    bits = ctypes.c_uint32(0)
    st = lib().mla_read_device_error(_ptr(dev_error), ctypes.byref(bits), _stream(stream))
    if st not in (MLA_OK, MLA_ERR_DEVICE_FAULT):
        _check("mla_read_device_error", st)
    return int(bits.value)


def mla_debug_wait_timeout(dev_error: torch.Tensor, timeout_ns: int, stream=None) -> None:
    _check("mla_debug_wait_timeout", lib().mla_debug_wait_timeout(_ptr(dev_error), int(timeout_ns), _stream(stream)))


# --------------------------------------------------------------------------- one decode step

def _check_table_rows(seq_lens, block_table) -> None:
    """Every page of every sequence needs an entry in its block-table row."""
    if block_table is None or block_table.dim() != 2:
        return
    pages = (np.asarray(seq_lens, dtype=np.int64) + PAGE - 1) // PAGE
    if pages.size and int(pages.max()) > int(block_table.shape[1]):
        raise ValueError(f"block_table rows hold {int(block_table.shape[1])} pages, a sequence needs "
                         f"{int(pages.max())}")


_sms = {}


def num_sms(device=None) -> int:
    index = torch.cuda.current_device() if device is None else device if isinstance(device, int) else torch.device(device).index
    if index is None:
        index = torch.cuda.current_device()
    if index not in _sms:
        _sms[index] = torch.cuda.get_device_properties(index).multi_processor_count
    return _sms[index]


class DecodeStep:
    """Device buffers and plan for one batch shape; ``run`` enqueues the step's kernels.

    absorb (q_c -> q_abs) -> paged decode (-> o_lat, lse, split partials) -> split merge -> W_UV
    projection (-> out), each a kernel of its own, chained by programmatic dependent launch (the
    measured fastest order at every workload of the benchmark).  fused_absorb runs the absorb as
    the bf16 decode kernel's prologue (mla_absorb_decode_paged); fused_tail runs merge and
    projection as one kernel (mla_merge_out_proj).  All buffers are allocated here, by torch, once.
    w_uk and w_uv may be 4-bit weights (W4Weight): the absorb and the projection are then
    mla_absorb_q_w4 and mla_out_proj_w4 (not with the fused kernels, nor from host memory; faster
    than bf16 up to some 30 rows of the batch, slower beyond 64).  With
    ``rope``, run_tokens takes the new tokens as their projections give them.  With ``window`` = W > 0
    a token sees the last W tokens up to itself and the first ``sinks``; pages without such a token
    are not read, and their table entries may hold anything.  With ``prefix`` the sequences begin
    with that shared prefix: seq_lens, block_table and the cache's rows are those of their own tokens
    behind it (at least one each; positions count the prefix), and the step ends with
    mla_prefix_attend, which joins both parts in out and lse (o_lat is the own tokens' alone).
    """

    def __init__(self, seq_lens, *, w_uk, w_uv, kv_pool: torch.Tensor,
                 block_table: torch.Tensor, kv_scale: Optional[torch.Tensor] = None,
                 kr_pool: Optional[torch.Tensor] = None, device=None, min_pages_per_split: int = 0,
                 max_clusters: int = 0, wait_timeout_ns: int = 0, item_cost_pages: int = 0,
                 softmax_scale: float = SOFTMAX_SCALE, fused_absorb: bool = False, fused_tail: bool = False,
                 queries_per_seq: int = 1, rope: Optional[Rope] = None, window: int = 0, sinks: int = 0,
                 prefix: Optional[SharedPrefix] = None):
        if prefix is not None and window:
            raise ValueError("prefix: a shared prefix is seen whole, a window is not supported with it")
        if (fused_absorb and isinstance(w_uk, W4Weight)) or (fused_tail and isinstance(w_uv, W4Weight)):
            raise ValueError("4-bit weights: the fused kernels read bf16 weights")
        if rope is not None and rope.dim != D_R:
            raise ValueError(f"rope: the step rotates {D_R} elements, got {rope.dim}")
        self.device = torch.device(device if device is not None else "cuda")
        self.seq_lens = np.asarray(seq_lens, dtype=np.int32)
        self.num_seqs = int(self.seq_lens.size)
        self.queries_per_seq = max(1, int(queries_per_seq))
        # query rows: token t of sequence b is row b * q + t (q_c, q_r, q_abs, o_lat, lse, out)
        self.batch = self.num_seqs * self.queries_per_seq
        self._plan_opts = dict(min_pages_per_split=min_pages_per_split, max_clusters=max_clusters,
                               wait_timeout_ns=wait_timeout_ns, item_cost_pages=item_cost_pages,
                               queries_per_seq=self.queries_per_seq, window=_i32(window), sinks=_i32(sinks))
        self._num_sms = num_sms(self.device)
        self.plan_host, self.info = mla_plan_splits(self.seq_lens, self._num_sms, **self._plan_opts)
        self.plan_dev = torch.from_numpy(self.plan_host).to(self.device)
        self._plan_info = self.info  # of the plan that run takes; info is that of the last step, run_host's too
        self.w_uk, self.w_uv = w_uk, w_uv
        self.kv_pool, self.kv_scale, self.kr_pool = kv_pool, kv_scale, kr_pool
        self.block_table = block_table
        _check_table_rows(self.seq_lens, block_table)
        self.softmax_scale = softmax_scale
        self.fused_absorb, self.fused_tail = bool(fused_absorb), bool(fused_tail)
        B = self.batch
        ws = int(self.info.workspace_bytes)
        self.workspace = torch.empty(max(ws // 4, 4), dtype=torch.float32, device=self.device) if ws else None
        self.q_abs = torch.empty(B, NUM_HEADS, D_C, dtype=torch.bfloat16, device=self.device)
        self.o_lat = torch.empty(B, NUM_HEADS, D_C, dtype=torch.bfloat16, device=self.device)
        self.lse = torch.empty(B, NUM_HEADS, dtype=torch.float32, device=self.device)
        self.out = torch.empty(B, NUM_HEADS, D_HC, dtype=torch.bfloat16, device=self.device)
        self.dev_error = torch.zeros(1, dtype=torch.int32, device=self.device)
        self.absorb_sync = torch.zeros(2, dtype=torch.int32, device=self.device)  # absorb-in-decode job counter
        self.rope = rope
        if rope is not None:  # the split and rotated queries of run_tokens
            self.q_c = torch.empty(B, NUM_HEADS, D_HC, dtype=torch.bfloat16, device=self.device)
            self.q_r = torch.empty(B, NUM_HEADS, D_R, dtype=torch.bfloat16, device=self.device)
        self.prefix = prefix
        self.prefix_workspace = None if prefix is None else prefix.workspace(B)
        self._host_workspace = self.workspace  # run_host's: a larger one where its lengths need it
        self._h_stage = self._d_stage = None  # pinned host / device staging of run_host
        self._host_graph = None  # (mla_step_graph handle, key of the buffers and lengths it was made for)

    def run(self, q_c: torch.Tensor, q_r: torch.Tensor, stream=None) -> torch.Tensor:
        kv = dict(kv_pool=self.kv_pool, block_table=self.block_table, o_lat=self.o_lat, lse=self.lse,
                  dev_error=self.dev_error, workspace=self.workspace, kv_scale=self.kv_scale, kr_pool=self.kr_pool,
                  softmax_scale=self.softmax_scale, stream=stream)
        if self.fused_absorb:
            mla_absorb_decode_paged(self._plan_info, self.plan_dev, q_c, self.w_uk, self.q_abs, self.absorb_sync, q_r, **kv)
        else:
            absorb = mla_absorb_q_w4 if isinstance(self.w_uk, W4Weight) else mla_absorb_q
            absorb(q_c, self.w_uk, self.q_abs, stream)
            mla_decode_paged(self._plan_info, self.plan_dev, self.q_abs, q_r, **kv)
        if self.fused_tail:
            mla_merge_out_proj(self._plan_info, self.plan_dev, self.workspace, self.o_lat, self.lse, self.w_uv, self.out,
                               self.dev_error, stream)
        else:
            mla_combine_splits(self._plan_info, self.plan_dev, self.workspace, self.o_lat, self.lse, stream)
            project = mla_out_proj_w4 if isinstance(self.w_uv, W4Weight) else mla_out_proj
            project(self.o_lat, self.w_uv, self.out, stream)
        if self.prefix is not None:
            mla_prefix_attend(self.prefix, q_c, q_r, self.out, lse=self.lse, own_out=self.out, own_lse=self.lse,
                              workspace=self.prefix_workspace, dev_error=self.dev_error,
                              softmax_scale=self.softmax_scale, stream=stream)
        return self.out

    def run_tokens(self, q: torch.Tensor, c_kv: torch.Tensor, k_r: torch.Tensor, positions: torch.Tensor,
                   slots: torch.Tensor, stream=None) -> torch.Tensor:
        """The step from the new tokens' projections: their rows into the cache with the keys
        rotated, their queries q [rows, 128, 192] split and rotated (mla_rope_append_kv, one
        launch), then ``run``.  Row b * queries_per_seq + t is new token t of sequence b, whose
        length counts it; slots and positions are its place in the pool and in the sequence."""
        if self.rope is None:
            raise ValueError("run_tokens: construct the step with rope=")
        if tuple(slots.shape) != (self.batch,):
            raise ValueError(f"run_tokens: expected {self.batch} tokens, got slots {tuple(slots.shape)}")
        if q is None:
            raise ValueError("run_tokens: q is needed")
        mla_rope_append_kv(self.rope, c_kv, k_r, positions, slots, kv_pool=self.kv_pool, kv_scale=self.kv_scale,
                           kr_pool=self.kr_pool, dev_error=self.dev_error, q=q, q_c=self.q_c, q_r=self.q_r,
                           stream=stream)
        return self.run(self.q_c, self.q_r, stream)

    @staticmethod
    def _host_key(q_c, q_r, block_table, lens, out):
        bt = None if block_table is None else (block_table.data_ptr(), tuple(block_table.shape), block_table.dtype)
        return (lens.tobytes(), q_c.data_ptr(), q_c.numel(), q_c.dtype, q_r.data_ptr(), q_r.numel(), q_r.dtype, bt,
                out.data_ptr(), out.numel(), out.dtype)

    def _drop_host_graph(self) -> None:
        if self._host_graph is not None:
            handle, self._host_graph = self._host_graph[0], None
            lib().mla_step_graph_destroy(handle)

    def __del__(self):
        try:
            self._drop_host_graph()
        except Exception:
            pass

    def run_host(self, q_c: torch.Tensor, q_r: torch.Tensor, *, block_table: Optional[torch.Tensor] = None,
                 seq_lens=None, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """One decode step from host (CPU) tensors, end to end: plan on the host for ``seq_lens``
        (the lengths given at construction when None; same batch size), copy the block table (a
        CPU int32 [batch, max_pages] tensor, when given; otherwise the device table given at
        construction is used) and the queries to the device, run the four kernels, and copy the
        result into ``out`` (a CPU bf16 [batch, 128, 128] tensor, pinned and allocated once if not
        given).  Returns ``out`` once the stream is done.

        When ``out``, the queries and the table are all pinned, the step is captured once as a
        CUDA graph (``mla_step_graph_create``: the plan is copied to the device at capture) and
        later calls with the same tensors and lengths only launch it (``mla_step_graph_run``),
        so a serving loop that writes each step's queries into the same pinned tensors pays for
        the copies and kernels only.  Otherwise each call is one ``mla_decode_step_host``."""
        if isinstance(self.w_uk, W4Weight) or isinstance(self.w_uv, W4Weight):
            raise ValueError("run_host: the step from host memory reads bf16 weights")
        if self.prefix is not None:
            raise ValueError("run_host: the step from host memory takes no shared prefix")
        lens = self.seq_lens if seq_lens is None else np.ascontiguousarray(np.asarray(seq_lens, dtype=np.int32))
        if self._host_graph is not None and out is not None:
            if self._host_key(q_c, q_r, block_table, lens, out) == self._host_graph[1]:
                _check("mla_step_graph_run", lib().mla_step_graph_run(self._host_graph[0], 1, _stream(stream)))
                return out
        before = self._host_graph
        try:
            return self._run_host(q_c, q_r, block_table, lens, out, stream)
        finally:  # a graph that was replaced, or that no later call can use, goes behind its successor
            if before is not None and self._host_graph is not before:
                lib().mla_step_graph_destroy(before[0])

    def _run_host(self, q_c, q_r, block_table, lens, out, stream) -> torch.Tensor:
        """run_host where no captured step fits; the graph that was there is let go of (None) once its
        lengths or buffers are not the step's any more."""
        B = self.batch
        _need(q_c, "q_c", torch.bfloat16, (B, NUM_HEADS, D_HC), device=False)
        _need(q_r, "q_r", torch.bfloat16, (B, NUM_HEADS, D_R), device=False)
        if lens.size != self.num_seqs:
            raise ValueError("run_host: seq_lens must keep the number of sequences")
        if block_table is not None:
            _need(block_table, "block_table", torch.int32, device=False)
            if block_table.dim() != 2 or block_table.shape[0] != self.num_seqs:
                raise ValueError("block_table must be [sequences, max_pages]")
        if not np.array_equal(lens, self.seq_lens) or self._h_stage is None:
            # new lengths: size the workspace for their plan (the library plans again itself)
            self._host_graph = None
            self.seq_lens = lens.copy()
            _, info = mla_plan_splits(lens, self._num_sms, **self._plan_opts)
            ws = int(info.workspace_bytes)
            if ws and (self._host_workspace is None or self._host_workspace.numel() * 4 < ws):
                # (beside run's, whose address a graph of capture() holds)
                self._host_workspace = torch.empty(ws // 4, dtype=torch.float32, device=self.device)
            if self._h_stage is None:
                cap = int(lib().mla_plan_bytes_max(B, self._num_sms))
                self._h_stage = torch.empty(cap // 4, dtype=torch.int32).pin_memory()
                self._d_stage = torch.empty(cap // 4, dtype=torch.int32, device=self.device)
                self._q_c_dev = torch.empty(B, NUM_HEADS, D_HC, dtype=torch.bfloat16, device=self.device)
                self._q_r_dev = torch.empty(B, NUM_HEADS, D_R, dtype=torch.bfloat16, device=self.device)
        if block_table is not None and (getattr(self, "_bt_dev", None) is None or
                                        tuple(self._bt_dev.shape) != tuple(block_table.shape)):
            self._host_graph = None
            self._bt_dev = torch.empty(tuple(block_table.shape), dtype=torch.int32, device=self.device)
        bt_dev = self._bt_dev if block_table is not None else self.block_table
        _check_table_rows(lens, bt_dev)
        use_graph = out is not None and q_c.is_pinned() and q_r.is_pinned() and out.is_pinned() and \
            (block_table is None or block_table.is_pinned())
        if out is None:
            out = torch.empty(B, NUM_HEADS, D_HC, dtype=torch.bfloat16).pin_memory()
        _need(out, "out", torch.bfloat16, (B, NUM_HEADS, D_HC), device=False)
        dtype = MLA_KV_BF16 if self.kv_scale is None else MLA_KV_FP8_E4M3
        bufs = StepBuffers(_addr(self._q_c_dev), _addr(self._q_r_dev), _addr(self.q_abs), _addr(bt_dev),
                           _addr(self._d_stage), _addr(self._host_workspace),
                           0 if self._host_workspace is None else self._host_workspace.numel() * 4, _addr(self.o_lat),
                           _addr(self.lse), _addr(self.out), _addr(self.dev_error), _addr(self._h_stage),
                           self._h_stage.numel() * 4)
        opts = PlanOptions(int(self._plan_opts["min_pages_per_split"]), int(self._plan_opts["max_clusters"]),
                           int(self._plan_opts["wait_timeout_ns"]), int(self._plan_opts["item_cost_pages"]),
                           self.queries_per_seq, int(self._plan_opts["window"]), int(self._plan_opts["sinks"]))
        info = PlanInfo()
        args = (lens.ctypes.data_as(ctypes.c_void_p), self.num_seqs, self._num_sms, ctypes.byref(opts), _ptr(q_c), _ptr(q_r),
                _ptr(block_table), int(bt_dev.shape[1]), _ptr(self.w_uk), _ptr(self.w_uv), dtype, _ptr(self.kv_pool),
                _ptr(self.kv_scale), _ptr(self.kr_pool), int(self.kv_pool.shape[0]), float(self.softmax_scale),
                ctypes.byref(bufs), _ptr(out), ctypes.byref(info), _stream(stream))
        if use_graph:
            self._host_graph = None
            handle = ctypes.c_void_p()
            _check("mla_step_graph_create", lib().mla_step_graph_create(*args, ctypes.byref(handle)))
            self._host_graph = (handle, self._host_key(q_c, q_r, block_table, lens, out))
            self.info = info
            _check("mla_step_graph_run", lib().mla_step_graph_run(handle, 1, _stream(stream)))
            return out
        _check("mla_decode_step_host", lib().mla_decode_step_host(*args))
        self.info = info
        return out

    def capture(self, q_c: torch.Tensor, q_r: torch.Tensor) -> "torch.cuda.CUDAGraph":
        """Capture one step into a CUDA graph and return it.

        The graph holds the step's kernels with their programmatic dependencies, reading
        ``q_c`` / ``q_r`` and writing ``self.out`` at their current addresses: copy the next
        step's queries into those tensors and call ``replay()`` (it runs on the current stream).
        The lengths, block table and cache are those of this object and stay fixed in the graph
        (a new plan needs a new capture).  One step runs eagerly first so that one-time set-up
        stays out of the capture."""
        self.run(q_c, q_r)
        torch.cuda.synchronize(self.device)
        try:  # keep the captured graph so that its nodes can be counted
            graph, kept = torch.cuda.CUDAGraph(keep_graph=True), True
        except TypeError:
            graph, kept = torch.cuda.CUDAGraph(), False
        with torch.cuda.graph(graph):
            self.run(q_c, q_r)
        self.graph_kernel_nodes = None
        if kept:
            try:
                self.graph_kernel_nodes = graph_kernel_nodes(graph.raw_cuda_graph())
            except (OSError, AttributeError, RuntimeError):
                self.graph_kernel_nodes = None
            graph.instantiate()
        return graph

    def device_error(self, stream=None) -> int:
        return mla_read_device_error(self.dev_error, stream)

    @property
    def launches_per_step(self) -> int:
        # the absorb runs inside the bf16 decode kernel when fused (a kernel of its own with the e4m3
        # cache); the merge is skipped when no sequence is split
        n = 1 if (self.fused_absorb and self.kv_scale is None) else 2
        n += 2 if self.prefix is not None else 0
        if self.fused_tail:
            return n + 1
        return n + 1 + (1 if self._plan_info.num_combine > 0 else 0)


def graph_kernel_nodes(raw_graph: int) -> int:
    """Number of kernel nodes in a CUDA graph (driver API, read only)."""
    cu = ctypes.CDLL("libcuda.so.1")
    n = ctypes.c_size_t(0)
    if cu.cuGraphGetNodes(ctypes.c_void_p(raw_graph), None, ctypes.byref(n)) != 0:
        raise RuntimeError("cuGraphGetNodes failed")
    nodes = (ctypes.c_void_p * n.value)()
    if n.value and cu.cuGraphGetNodes(ctypes.c_void_p(raw_graph), nodes, ctypes.byref(n)) != 0:
        raise RuntimeError("cuGraphGetNodes failed")
    kernels = 0
    for i in range(n.value):
        t = ctypes.c_int(-1)
        if cu.cuGraphNodeGetType(ctypes.c_void_p(nodes[i]), ctypes.byref(t)) != 0:
            raise RuntimeError("cuGraphNodeGetType failed")
        kernels += int(t.value == 0)  # CU_GRAPH_NODE_TYPE_KERNEL
    return kernels


def inputs_to_device(inp, device="cuda"):
    """Move a synth.DecodeInputs to the device: (q_c, q_r, w_uk, w_uv, kv dict, block_table)."""
    dev = torch.device(device)
    kv = {}
    if inp.kv_dtype == "bf16":
        kv["kv_pool"] = inp.pool.to(dev)
    else:
        kv["kv_pool"] = inp.c8.to(dev)
        kv["kv_scale"] = inp.kv_scale.to(dev)
        kv["kr_pool"] = inp.kr.to(dev)
    bt = torch.from_numpy(np.ascontiguousarray(inp.block_table)).to(dev)
    return inp.q_c.to(dev), inp.q_r.to(dev), inp.w_uk.to(dev), inp.w_uv.to(dev), kv, bt
