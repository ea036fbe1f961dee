"""Python binding of libmok (the MI355X MoE-layer library).

Argument marshalling only: every step of the layer runs in the HIP kernels of
``libmok.so``; PyTorch provides device memory and the stream. Importing this
package raises if the library has not been built
(``python mixture_experts_layer_table_amd/build.py``).

Two levels, after the pages' ops / functional split ("Mixture-of-Kittens (MoK)"
project summary, Functional API and Key-concepts table):

* ``mok_*`` — one function per C-ABI entry point, same names and arguments;
  tensors are passed as raw pointers and the caller owns every buffer.
* ``MoKConfig``, ``get_workspace``, ``build_schedule``, ``forward``,
  ``backward``, ``mxfp8_quantize`` — allocate the caller-side buffers with
  torch and call the entry points above. Around the layer: ``dropout``,
  ``add_rmsnorm``, ``get_ffn_workspace``, ``ffn_forward`` and their backwards.
  The routed experts taken apart: ``sort_tokens``, ``permute``, ``unpermute`` and
  their backwards, ``fp8_quantize``, ``glu_backward``, ``fp8_matmul``,
  ``fp8_wgrad``.
"""
from __future__ import annotations

import ctypes
import dataclasses
import functools
import os

__version__ = "0.1.0"

# Device memory and streams come from PyTorch, so the library must run on the
# HIP runtime torch has loaded: import torch first, so that libmok's dependency
# on libamdhip64.so.7 resolves to that same copy instead of a second runtime.
import torch  # noqa: E402,F401

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmok.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(f"{_LIB_PATH} is missing: build it with "
                      "`python mixture_experts_layer_table_amd/build.py` (there is no fallback)")
_lib = ctypes.CDLL(_LIB_PATH)

MOK_OK, MOK_ERROR_INVALID_VALUE, MOK_ERROR_UNSUPPORTED, MOK_ERROR_BUFFER_TOO_SMALL, \
    MOK_ERROR_LAUNCH_FAILED = range(5)
MOK_BF16, MOK_MXFP8, MOK_MXFP8_WGRAD = 0, 1, 2
MOK_SCHEDULE_OVERFLOW, MOK_BAD_EXPERT_ID, MOK_SCHEDULER_STALLED, MOK_SCHEDULE_MISMATCH = 1, 2, 4, 8
MOK_DEBUG_IDENTITY_EXPERT, MOK_DEBUG_SEPARATE_LAUNCHES, MOK_DEBUG_WHOLE_PASS, MOK_DEBUG_FORCE_STALL = 1, 2, 4, 8

EXPORTS = ("mok_config_default", "mok_config_autosize", "mok_query_sizes", "mok_schedule_layout_query",
           "mok_build_schedule", "mok_forward", "mok_backward", "mok_mxfp8_quantize", "mok_route",
           "mok_route_backward", "mok_status_string", "mok_kernel_timing_enable", "mok_kernel_timing_read",
           "mok_last_error", "mok_forward_noalloc", "mok_item_trace_enable", "mok_item_trace_read",
           "mok_dropout", "mok_dropout_backward", "mok_add_rmsnorm", "mok_add_rmsnorm_backward_size",
           "mok_add_rmsnorm_backward", "mok_ffn_query_size", "mok_ffn_forward", "mok_ffn_backward",
           "mok_sort_tokens_size", "mok_sort_tokens", "mok_permute", "mok_permute_backward", "mok_unpermute",
           "mok_unpermute_backward", "mok_fp8_quantize", "mok_glu_backward", "mok_fp8_matmul_size", "mok_fp8_matmul",
           "mok_fp8_wgrad_size", "mok_fp8_wgrad")
MOK_TRACE_FWD_GEMMS, MOK_TRACE_BWD_GEMMS, MOK_TRACE_WGRAD_GATE_UP, MOK_TRACE_WGRAD_DOWN, MOK_TRACE_OTHER = range(5)
MOK_ITEM_TRACE_CAPACITY = 65536
MOK_NOALLOC_SCRATCH_BYTES = 64 << 20
MOK_STREAM_BF16, MOK_STREAM_F32 = 0, 1
MOK_FP8_TURNED, MOK_FP8_TILE, MOK_FP8_GLU = 1, 2, 4


class mok_config(ctypes.Structure):
    _fields_ = [("minibatch_rows", ctypes.c_int32), ("precision", ctypes.c_int32),
                ("macrobatch_tokens", ctypes.c_int64), ("ring_bytes", ctypes.c_int64),
                ("capacity_multiplier", ctypes.c_float), ("debug_flags", ctypes.c_uint32),
                ("persistent_workgroups", ctypes.c_int32)]


class mok_shape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int32), ("I", ctypes.c_int32),
                ("E", ctypes.c_int32), ("k", ctypes.c_int32)]


class mok_weights(ctypes.Structure):
    _fields_ = [("w_gate", ctypes.c_void_p), ("w_up", ctypes.c_void_p), ("w_down", ctypes.c_void_p),
                ("gate_elems", ctypes.c_void_p), ("gate_scales", ctypes.c_void_p),
                ("up_elems", ctypes.c_void_p), ("up_scales", ctypes.c_void_p),
                ("down_elems", ctypes.c_void_p), ("down_scales", ctypes.c_void_p)]


class mok_norm_shape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int32), ("stream_dtype", ctypes.c_int32),
                ("eps", ctypes.c_float), ("p", ctypes.c_float)]


class mok_ffn_shape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int32), ("I", ctypes.c_int32),
                ("precision", ctypes.c_int32)]


class mok_sort_shape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("k", ctypes.c_int32), ("E", ctypes.c_int32), ("align", ctypes.c_int32)]


class mok_rows_shape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("rows", ctypes.c_int64), ("k", ctypes.c_int32), ("E", ctypes.c_int32),
                ("H", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class mok_fp8_shape(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("E", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32)]


class mok_kernel_stat(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 32), ("launches", ctypes.c_int64), ("total_ms", ctypes.c_double),
                ("max_ms", ctypes.c_double)]


class mok_item_record(ctypes.Structure):
    _fields_ = [("t_claim", ctypes.c_uint64), ("t_start", ctypes.c_uint64), ("t_kloop", ctypes.c_uint64),
                ("t_end", ctypes.c_uint64), ("launch", ctypes.c_uint32), ("kernel", ctypes.c_uint8),
                ("item_class", ctypes.c_uint8), ("xcd", ctypes.c_uint16), ("item", ctypes.c_uint32),
                ("workgroup", ctypes.c_uint32)]


class mok_schedule_layout(ctypes.Structure):
    _fields_ = [("R", ctypes.c_int64), ("NM", ctypes.c_int64), ("G", ctypes.c_int64),
                ("cap", ctypes.c_int64)] + \
        [(n, ctypes.c_size_t) for n in ("status", "n_seg", "counts", "offsets", "mcounts", "moffsets",
                                       "perm", "inv", "canon", "mb_start", "segments", "total_bytes")]


_P = ctypes.c_void_p
_sz = ctypes.POINTER(ctypes.c_size_t)
_sigs = {
    "mok_config_default": [ctypes.POINTER(mok_config)],
    "mok_config_autosize": [ctypes.POINTER(mok_config), ctypes.POINTER(mok_shape), ctypes.c_int32],
    "mok_query_sizes": [ctypes.POINTER(mok_config), ctypes.POINTER(mok_shape), _sz, _sz, _sz],
    "mok_schedule_layout_query": [ctypes.POINTER(mok_config), ctypes.POINTER(mok_shape),
                                  ctypes.POINTER(mok_schedule_layout)],
    "mok_build_schedule": [ctypes.POINTER(mok_config), ctypes.POINTER(mok_shape), _P, _P,
                           ctypes.c_size_t, _P],
    "mok_forward": [ctypes.POINTER(mok_config), ctypes.POINTER(mok_shape), _P, ctypes.c_size_t, _P,
                    ctypes.c_size_t, _P, _P, ctypes.POINTER(mok_weights), _P, _P, ctypes.c_size_t, _P],
    "mok_backward": [ctypes.POINTER(mok_config), ctypes.POINTER(mok_shape), _P, ctypes.c_size_t, _P,
                     ctypes.c_size_t, _P, _P, ctypes.POINTER(mok_weights), _P, ctypes.c_size_t, _P, _P, _P,
                     _P, _P, _P, _P],
    "mok_forward_noalloc": [ctypes.POINTER(mok_config), ctypes.POINTER(mok_shape), _P, ctypes.c_size_t, _P, _P,
                            ctypes.POINTER(mok_weights), _P, _P, ctypes.c_size_t, _P],
    "mok_mxfp8_quantize": [_P, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int32,
                           _P, _P, _P],
    "mok_route": [_P, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, _P, _P, _P],
    "mok_route_backward": [_P, _P, _P, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, _P, _P],
    "mok_dropout": [_P, _P, ctypes.c_int64, ctypes.c_float, _P, ctypes.c_int32, _P, _P],
    "mok_dropout_backward": [_P, ctypes.c_int64, ctypes.c_float, _P, ctypes.c_int32, _P, _P],
    "mok_add_rmsnorm": [ctypes.POINTER(mok_norm_shape), _P, _P, _P, _P, _P, _P, _P, _P, _P, _P],
    "mok_add_rmsnorm_backward_size": [ctypes.POINTER(mok_norm_shape), _sz],
    "mok_add_rmsnorm_backward": [ctypes.POINTER(mok_norm_shape), _P, ctypes.c_size_t, _P, _P, _P, _P, _P, _P, _P,
                                 _P, _P, _P],
    "mok_ffn_query_size": [ctypes.POINTER(mok_ffn_shape), _sz],
    "mok_ffn_forward": [ctypes.POINTER(mok_ffn_shape), _P, ctypes.c_size_t, _P, _P, _P,
                        ctypes.POINTER(mok_weights), _P, _P, _P, _P],
    "mok_ffn_backward": [ctypes.POINTER(mok_ffn_shape), _P, ctypes.c_size_t, _P, ctypes.POINTER(mok_weights), _P, _P,
                         _P, _P, _P, _P, _P, _P],
    "mok_sort_tokens_size": [ctypes.POINTER(mok_sort_shape), ctypes.POINTER(ctypes.c_int64), _sz],
    "mok_sort_tokens": [ctypes.POINTER(mok_sort_shape), _P, ctypes.c_size_t, _P, _P, _P, _P, _P],
    "mok_permute": [ctypes.POINTER(mok_rows_shape), _P, _P, _P, _P, _P, _P, _P, _P],
    "mok_permute_backward": [ctypes.POINTER(mok_rows_shape), _P, _P, _P, _P],
    "mok_unpermute": [ctypes.POINTER(mok_rows_shape), _P, _P, _P, _P, _P, _P],
    "mok_unpermute_backward": [ctypes.POINTER(mok_rows_shape), _P, _P, _P, _P, _P, _P, _P, _P, _P],
    "mok_fp8_quantize": [_P, ctypes.c_int32, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_uint32, _P, _P,
                         _P],
    "mok_glu_backward": [_P, _P, ctypes.c_int64, ctypes.c_int32, _P, _P],
    "mok_fp8_matmul_size": [ctypes.POINTER(mok_fp8_shape), _sz],
    "mok_fp8_matmul": [ctypes.POINTER(mok_fp8_shape), _P, ctypes.c_size_t, _P, _P, _P, _P, _P, _P, _P],
    "mok_fp8_wgrad_size": [ctypes.POINTER(mok_fp8_shape), _sz],
    "mok_fp8_wgrad": [ctypes.POINTER(mok_fp8_shape), _P, ctypes.c_size_t, _P, _P, _P, _P, _P, _P, _P, _P],
    "mok_kernel_timing_enable": [ctypes.c_int32],
    "mok_item_trace_enable": [ctypes.c_int32],
    "mok_item_trace_read": [ctypes.POINTER(mok_item_record), ctypes.c_int32, ctypes.POINTER(ctypes.c_int32)],
    "mok_kernel_timing_read": [ctypes.POINTER(mok_kernel_stat), ctypes.c_int32, ctypes.POINTER(ctypes.c_int32)],
}
for _name, _args in _sigs.items():
    _f = getattr(_lib, _name)
    _f.argtypes = _args
    _f.restype = ctypes.c_int
_lib.mok_status_string.argtypes = [ctypes.c_int]
_lib.mok_status_string.restype = ctypes.c_char_p
_lib.mok_last_error.argtypes = []
_lib.mok_last_error.restype = ctypes.c_char_p


class MokError(RuntimeError):
    def __init__(self, status: int, where: str):
        detail = mok_last_error() if status == MOK_ERROR_LAUNCH_FAILED else ""
        super().__init__(f"{where}: {mok_status_string(status)}" + (f" ({detail})" if detail else ""))
        self.status = status


def _check(status: int, where: str):
    if status != MOK_OK:
        raise MokError(status, where)


def mok_status_string(status: int) -> str:
    return _lib.mok_status_string(status).decode()


def mok_last_error() -> str:
    return _lib.mok_last_error().decode()


# ----------------------------------------------------------------------------- raw entry points

def mok_config_default(cfg):
    return _lib.mok_config_default(ctypes.byref(cfg))


def mok_config_autosize(cfg, shape, n_cu):
    return _lib.mok_config_autosize(ctypes.byref(cfg), ctypes.byref(shape), n_cu)


def mok_query_sizes(cfg, shape, workspace, schedule, fwd_ctx):
    return _lib.mok_query_sizes(ctypes.byref(cfg), ctypes.byref(shape), workspace, schedule, fwd_ctx)


def mok_schedule_layout_query(cfg, shape, layout):
    return _lib.mok_schedule_layout_query(ctypes.byref(cfg), ctypes.byref(shape), ctypes.byref(layout))


def mok_build_schedule(cfg, shape, topk_ids, schedule, schedule_bytes, stream):
    return _lib.mok_build_schedule(ctypes.byref(cfg), ctypes.byref(shape), topk_ids, schedule,
                                   schedule_bytes, stream)


def mok_forward(cfg, shape, schedule, schedule_bytes, workspace, workspace_bytes, x, topk_w, weights, out,
                fwd_ctx, fwd_ctx_bytes, stream):
    return _lib.mok_forward(ctypes.byref(cfg), ctypes.byref(shape), schedule, schedule_bytes, workspace,
                            workspace_bytes, x, topk_w, ctypes.byref(weights), out, fwd_ctx, fwd_ctx_bytes,
                            stream)


def mok_backward(cfg, shape, schedule, schedule_bytes, workspace, workspace_bytes, x, topk_w, weights,
                 fwd_ctx, fwd_ctx_bytes, dy, dx, dw_gate, dw_up, dw_down, dtopk_w, stream):
    return _lib.mok_backward(ctypes.byref(cfg), ctypes.byref(shape), schedule, schedule_bytes, workspace,
                             workspace_bytes, x, topk_w, ctypes.byref(weights), fwd_ctx, fwd_ctx_bytes,
                             dy, dx, dw_gate, dw_up, dw_down, dtopk_w, stream)


def mok_forward_noalloc(cfg, shape, schedule, schedule_bytes, x, topk_w, weights, out, fwd_ctx, fwd_ctx_bytes,
                        stream):
    return _lib.mok_forward_noalloc(ctypes.byref(cfg), ctypes.byref(shape), schedule, schedule_bytes, x, topk_w,
                                    ctypes.byref(weights), out, fwd_ctx, fwd_ctx_bytes, stream)


def mok_mxfp8_quantize(src, batch, rows, K, src_is_k_by_rows, elems, scales, stream):
    return _lib.mok_mxfp8_quantize(src, batch, rows, K, src_is_k_by_rows, elems, scales, stream)


def mok_route(logits, T, E, k, topk_ids, topk_w, stream):
    return _lib.mok_route(logits, T, E, k, topk_ids, topk_w, stream)


def mok_route_backward(topk_ids, topk_w, dtopk_w, T, E, k, dlogits, stream):
    return _lib.mok_route_backward(topk_ids, topk_w, dtopk_w, T, E, k, dlogits, stream)


def mok_dropout(x, residual, n, p, rng, stream_dtype, out, stream):
    return _lib.mok_dropout(x, residual, n, p, rng, stream_dtype, out, stream)


def mok_dropout_backward(dy, n, p, rng, stream_dtype, dx, stream):
    return _lib.mok_dropout_backward(dy, n, p, rng, stream_dtype, dx, stream)


def mok_add_rmsnorm(shape, x, residual, weight, rng, sum, y, y_elems, y_scales, rstd, stream):
    return _lib.mok_add_rmsnorm(ctypes.byref(shape), x, residual, weight, rng, sum, y, y_elems, y_scales, rstd, stream)


def mok_add_rmsnorm_backward_size(shape, workspace):
    return _lib.mok_add_rmsnorm_backward_size(ctypes.byref(shape), workspace)


def mok_add_rmsnorm_backward(shape, workspace, workspace_bytes, dy, sum, weight, rstd, dsum, rng, dresidual, dx,
                             dweight, stream):
    return _lib.mok_add_rmsnorm_backward(ctypes.byref(shape), workspace, workspace_bytes, dy, sum, weight, rstd, dsum,
                                         rng, dresidual, dx, dweight, stream)


def mok_ffn_query_size(shape, workspace):
    return _lib.mok_ffn_query_size(ctypes.byref(shape), workspace)


def mok_ffn_forward(shape, workspace, workspace_bytes, x, x_elems, x_scales, weights, addend, out, h, stream):
    return _lib.mok_ffn_forward(ctypes.byref(shape), workspace, workspace_bytes, x, x_elems, x_scales,
                                ctypes.byref(weights), addend, out, h, stream)


def mok_ffn_backward(shape, workspace, workspace_bytes, x, weights, h, dy, addend, dx, dw_gate, dw_up, dw_down,
                     stream):
    return _lib.mok_ffn_backward(ctypes.byref(shape), workspace, workspace_bytes, x, ctypes.byref(weights), h, dy,
                                 addend, dx, dw_gate, dw_up, dw_down, stream)


def mok_sort_tokens_size(shape, rows, workspace):
    return _lib.mok_sort_tokens_size(ctypes.byref(shape), rows, workspace)


def mok_sort_tokens(shape, workspace, workspace_bytes, topk_ids, offsets, slots, row_slots, stream):
    return _lib.mok_sort_tokens(ctypes.byref(shape), workspace, workspace_bytes, topk_ids, offsets, slots, row_slots,
                                stream)


def mok_permute(shape, x, offsets, slots, row_slots, rows, elems, scales, stream):
    return _lib.mok_permute(ctypes.byref(shape), x, offsets, slots, row_slots, rows, elems, scales, stream)


def mok_permute_backward(shape, drows, slots, dx, stream):
    return _lib.mok_permute_backward(ctypes.byref(shape), drows, slots, dx, stream)


def mok_unpermute(shape, y, slots, w, addend, out, stream):
    return _lib.mok_unpermute(ctypes.byref(shape), y, slots, w, addend, out, stream)


def mok_unpermute_backward(shape, dout, y, offsets, slots, row_slots, w, dy, dw, stream):
    return _lib.mok_unpermute_backward(ctypes.byref(shape), dout, y, offsets, slots, row_slots, w, dy, dw, stream)


def mok_fp8_quantize(src, dtype, batch, rows, K, flags, elems, scales, stream):
    return _lib.mok_fp8_quantize(src, dtype, batch, rows, K, flags, elems, scales, stream)


def mok_glu_backward(da, h, T, I, dh, stream):
    return _lib.mok_glu_backward(da, h, T, I, dh, stream)


def mok_fp8_matmul_size(shape, workspace):
    return _lib.mok_fp8_matmul_size(ctypes.byref(shape), workspace)


def mok_fp8_matmul(shape, workspace, workspace_bytes, a_elems, a_scales, b_elems, b_scales, offsets, out, stream):
    return _lib.mok_fp8_matmul(ctypes.byref(shape), workspace, workspace_bytes, a_elems, a_scales, b_elems, b_scales,
                               offsets, out, stream)


def mok_fp8_wgrad_size(shape, workspace):
    return _lib.mok_fp8_wgrad_size(ctypes.byref(shape), workspace)


def mok_fp8_wgrad(shape, workspace, workspace_bytes, dy_elems, dy_scales, x_elems, x_scales, offsets, addend, out,
                  stream):
    return _lib.mok_fp8_wgrad(ctypes.byref(shape), workspace, workspace_bytes, dy_elems, dy_scales, x_elems, x_scales,
                              offsets, addend, out, stream)


def mok_kernel_timing_enable(enable):
    return _lib.mok_kernel_timing_enable(enable)


def mok_kernel_timing_read(stats, capacity, count):
    return _lib.mok_kernel_timing_read(stats, capacity, count)


def mok_item_trace_enable(enable):
    return _lib.mok_item_trace_enable(enable)


def mok_item_trace_read(records, capacity, count):
    return _lib.mok_item_trace_read(records, capacity, count)


def item_trace_read():
    """The per-item trace records so far as a numpy structured array (synchronises)."""
    import numpy as np
    cap = MOK_ITEM_TRACE_CAPACITY
    arr = (mok_item_record * cap)()
    n = ctypes.c_int32()
    _check(mok_item_trace_read(arr, cap, ctypes.byref(n)), "mok_item_trace_read")
    dt = np.dtype([("t_claim", "<u8"), ("t_start", "<u8"), ("t_kloop", "<u8"), ("t_end", "<u8"),
                   ("launch", "<u4"), ("kernel", "u1"), ("item_class", "u1"), ("xcd", "<u2"),
                   ("item", "<u4"), ("workgroup", "<u4")])
    assert dt.itemsize == ctypes.sizeof(mok_item_record)
    buf = np.frombuffer(bytes(arr), dtype=dt)
    return buf[:min(n.value, cap)].copy(), n.value


def kernel_times(enable_after: bool = False):
    """Read (and clear) the per-kernel timing records: {name: (launches, total_ms, max_ms)}."""
    cap = 64
    arr = (mok_kernel_stat * cap)()
    n = ctypes.c_int32()
    _check(mok_kernel_timing_read(arr, cap, ctypes.byref(n)), "mok_kernel_timing_read")
    out = {arr[i].name.decode(): (arr[i].launches, arr[i].total_ms, arr[i].max_ms) for i in range(min(n.value, cap))}
    if not enable_after:
        _check(mok_kernel_timing_enable(0), "mok_kernel_timing_enable")
    return out


# ----------------------------------------------------------------------------- functional layer

@dataclasses.dataclass
class MoKConfig:
    """Layer knobs; none of them changes any output bit."""
    minibatch_rows: int = 512
    macrobatch_tokens: int = 0
    ring_bytes: int = 256 << 20
    capacity_multiplier: float = 1.0
    precision: int = MOK_BF16
    debug_flags: int = 0
    persistent_workgroups: int = 0      # 0: one per compute unit

    def c(self) -> mok_config:
        return mok_config(self.minibatch_rows, self.precision, self.macrobatch_tokens,
                          self.ring_bytes, self.capacity_multiplier, self.debug_flags,
                          self.persistent_workgroups)


def _shape(T, H, I, E, k) -> mok_shape:
    return mok_shape(T, H, I, E, k)


def autosize_config(config: MoKConfig, T, H, I, E, k, n_cu: int = 0) -> MoKConfig:
    """Copy of ``config`` with the mini-batch sized by the two-wave rule (mok_config_autosize)."""
    c = config.c()
    _check(mok_config_autosize(c, _shape(T, H, I, E, k), n_cu), "mok_config_autosize")
    return dataclasses.replace(config, minibatch_rows=c.minibatch_rows, ring_bytes=c.ring_bytes)


def query_sizes(config: MoKConfig, T, H, I, E, k):
    ws, sc, cx = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(mok_query_sizes(config.c(), _shape(T, H, I, E, k), ctypes.byref(ws), ctypes.byref(sc),
                           ctypes.byref(cx)), "mok_query_sizes")
    return ws.value, sc.value, cx.value


def schedule_layout(config: MoKConfig, T, H, I, E, k) -> mok_schedule_layout:
    lay = mok_schedule_layout()
    _check(mok_schedule_layout_query(config.c(), _shape(T, H, I, E, k), lay), "mok_schedule_layout_query")
    return lay


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _require(t, name, dtype, shape, device=None):
    """The C ABI receives raw pointers and no sizes for most tensors, so every
    tensor is checked here before a call: dtype (an int64 id tensor read as
    int32 would route silently wrong), exact shape (a short output would be
    written past its end), contiguity and device."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if device is not None and t.device != torch.device(device):
        raise ValueError(f"{name}: on {t.device}, expected {device}")


def _require_bytes(t, name, nbytes, device=None):
    """A caller-given uint8 buffer of at least nbytes (workspace, schedule, fwd_ctx)."""
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype != torch.uint8 or t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous 1-D uint8 tensor")
    if t.numel() < nbytes:
        raise ValueError(f"{name}: {t.numel()} bytes, need {nbytes}")
    if device is not None and t.device != torch.device(device):
        raise ValueError(f"{name}: on {t.device}, expected {device}")


def _stream():
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


@dataclasses.dataclass
class Workspace:
    """Caller-owned device buffers for one layer shape (made once, reused)."""
    config: MoKConfig
    T: int
    H: int
    I: int
    E: int
    k: int
    buffer: "object"        # torch.uint8 tensor
    schedule_bytes: int
    fwd_ctx_bytes: int


def get_workspace(config: MoKConfig, *, device, num_local_tokens: int, hidden_size: int,
                  intermediate_size: int, num_experts: int, topk: int) -> Workspace:
    import torch
    ws, sc, cx = query_sizes(config, num_local_tokens, hidden_size, intermediate_size, num_experts, topk)
    buf = torch.empty(max(ws, 256), dtype=torch.uint8, device=device)
    return Workspace(config, num_local_tokens, hidden_size, intermediate_size, num_experts, topk, buf,
                     sc, cx)


def build_schedule(ws: Workspace, topk_ids, schedule=None):
    """topk_ids: int32 [T,k] on the device. Returns the schedule buffer (uint8 tensor)."""
    import torch
    dev = ws.buffer.device
    _require(topk_ids, "topk_ids", torch.int32, (ws.T, ws.k), dev)
    if schedule is None:
        schedule = torch.empty(max(ws.schedule_bytes, 256), dtype=torch.uint8, device=dev)
    _require_bytes(schedule, "schedule", ws.schedule_bytes, dev)
    _check(mok_build_schedule(ws.config.c(), _shape(ws.T, ws.H, ws.I, ws.E, ws.k), _ptr(topk_ids),
                              _ptr(schedule), schedule.numel(), _stream()), "mok_build_schedule")
    return schedule


def weights_bf16(w_gate, w_up, w_down) -> mok_weights:
    """The struct keeps references to the tensors, so their memory lives as long as it does."""
    w = mok_weights(w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr(), None, None, None, None, None, None)
    w._tensors = (w_gate, w_up, w_down)
    w._kind = "bf16"
    return w


def weights_mxfp8(gate, up, down, orientation: str = "") -> mok_weights:
    """Each argument is an (elems, scales) pair of uint8 tensors (kept referenced
    by the struct); orientation "fwd" or "bwd" when known (MXFP8Weights sets it)."""
    w = mok_weights(None, None, None, gate[0].data_ptr(), gate[1].data_ptr(), up[0].data_ptr(),
                    up[1].data_ptr(), down[0].data_ptr(), down[1].data_ptr())
    w._tensors = (gate, up, down)
    w._kind = "mxfp8" + (":" + orientation if orientation else "")
    return w


def _check_weights(ws: "Workspace", weights: mok_weights, orientation: str):
    """Shapes, dtypes and devices of the tensors a weight struct refers to."""
    import torch
    tensors = getattr(weights, "_tensors", None)
    if tensors is None:          # a hand-made struct: nothing to check against
        return
    dev = ws.buffer.device
    E, H, I = ws.E, ws.H, ws.I
    mx = ws.config.precision in (MOK_MXFP8, MOK_MXFP8_WGRAD)
    kind = getattr(weights, "_kind", "")
    if not mx:
        if not kind.startswith("bf16"):
            raise ValueError("BF16 mode needs bf16 weights (weights_bf16)")
        for t, n, sh in zip(tensors, ("w_gate", "w_up", "w_down"), ((E, H, I), (E, H, I), (E, I, H))):
            _require(t, n, torch.bfloat16, sh, dev)
        return
    if not kind.startswith("mxfp8"):
        raise ValueError("MXFP8 mode needs quantized weights (MXFP8Weights)")
    if ":" in kind and kind.split(":")[1] != orientation:
        raise ValueError(f"MXFP8 weights quantized for {kind.split(':')[1]}, used in {orientation}")
    if orientation == "fwd":        # quantized along the forward contraction axes
        shapes = ((E, I, H), (E, I, H), (E, H, I))
    else:
        shapes = ((E, H, I), (E, H, I), (E, I, H))
    for (el, sc), n, sh in zip(tensors, ("gate", "up", "down"), shapes):
        _require(el, n + " elements", torch.uint8, sh, dev)
        _require(sc, n + " scales", torch.uint8, sh[:2] + (sh[2] // 32,), dev)


class MXFP8Weights:
    """Expert weights quantized once for MXFP8 mode, in both orientations the
    layer needs (quantized along the contraction axis of each GEMM):
    ``fwd`` for mok_forward (W_gate^T, W_up^T [E,I,H] along H; W_down^T
    [E,H,I] along I) and ``bwd`` for mok_backward (W_gate, W_up [E,H,I] along
    I; W_down [E,I,H] along H). Holds the uint8 tensors the pointers refer to."""

    def __init__(self, w_gate, w_up, w_down):
        self.fwd_gate = mxfp8_quantize(w_gate, True)
        self.fwd_up = mxfp8_quantize(w_up, True)
        self.fwd_down = mxfp8_quantize(w_down, True)
        self.bwd_gate = mxfp8_quantize(w_gate, False)
        self.bwd_up = mxfp8_quantize(w_up, False)
        self.bwd_down = mxfp8_quantize(w_down, False)
        self.fwd = weights_mxfp8(self.fwd_gate, self.fwd_up, self.fwd_down, "fwd")
        self.bwd = weights_mxfp8(self.bwd_gate, self.bwd_up, self.bwd_down, "bwd")


def forward(ws: Workspace, schedule, x, topk_w, weights: mok_weights, out=None, fwd_ctx=None):
    """Returns (out bf16 [T,H], fwd_ctx uint8)."""
    import torch
    dev = ws.buffer.device
    if out is None:
        out = torch.empty((ws.T, ws.H), dtype=torch.bfloat16, device=dev)
    if fwd_ctx is None:
        fwd_ctx = torch.empty(max(ws.fwd_ctx_bytes, 256), dtype=torch.uint8, device=dev)
    _require_bytes(schedule, "schedule", ws.schedule_bytes, dev)
    _require(x, "x", torch.bfloat16, (ws.T, ws.H), dev)
    _require(topk_w, "topk_w", torch.float32, (ws.T, ws.k), dev)
    _require(out, "out", torch.bfloat16, (ws.T, ws.H), dev)
    _require_bytes(fwd_ctx, "fwd_ctx", ws.fwd_ctx_bytes, dev)
    _check_weights(ws, weights, "fwd")
    _check(mok_forward(ws.config.c(), _shape(ws.T, ws.H, ws.I, ws.E, ws.k), _ptr(schedule),
                       schedule.numel(), _ptr(ws.buffer), ws.buffer.numel(), _ptr(x), _ptr(topk_w), weights, _ptr(out),
                       _ptr(fwd_ctx), fwd_ctx.numel(), _stream()), "mok_forward")
    return out, fwd_ctx


def forward_noalloc(ws: Workspace, schedule, x, topk_w, weights: mok_weights, out, fwd_ctx):
    """forward() through mok_forward_noalloc: the library's static scratch
    instead of ws.buffer (ws supplies the config and shape only). out and
    fwd_ctx are caller-given; nothing is allocated here or in the call."""
    import torch
    dev = ws.buffer.device
    _require_bytes(schedule, "schedule", ws.schedule_bytes, dev)
    _require(x, "x", torch.bfloat16, (ws.T, ws.H), dev)
    _require(topk_w, "topk_w", torch.float32, (ws.T, ws.k), dev)
    _require(out, "out", torch.bfloat16, (ws.T, ws.H), dev)
    _require_bytes(fwd_ctx, "fwd_ctx", ws.fwd_ctx_bytes, dev)
    _check_weights(ws, weights, "fwd")
    _check(mok_forward_noalloc(ws.config.c(), _shape(ws.T, ws.H, ws.I, ws.E, ws.k), _ptr(schedule),
                               schedule.numel(), _ptr(x), _ptr(topk_w), weights, _ptr(out), _ptr(fwd_ctx),
                               fwd_ctx.numel(), _stream()), "mok_forward_noalloc")
    return out, fwd_ctx


def backward(ws: Workspace, schedule, fwd_ctx, x, topk_w, weights: mok_weights, dy, grads=None):
    """Returns dict(dx, dw_gate, dw_up, dw_down, dtopk_w)."""
    import torch
    dev = ws.buffer.device
    shapes = dict(dx=((ws.T, ws.H), torch.bfloat16), dw_gate=((ws.E, ws.H, ws.I), torch.bfloat16),
                  dw_up=((ws.E, ws.H, ws.I), torch.bfloat16), dw_down=((ws.E, ws.I, ws.H), torch.bfloat16),
                  dtopk_w=((ws.T, ws.k), torch.float32))
    if grads is None:
        grads = {n: torch.empty(sh, dtype=dt, device=dev) for n, (sh, dt) in shapes.items()}
    for n, (sh, dt) in shapes.items():
        _require(grads[n], n, dt, sh, dev)
    _require_bytes(schedule, "schedule", ws.schedule_bytes, dev)
    _require_bytes(fwd_ctx, "fwd_ctx", ws.fwd_ctx_bytes, dev)
    _require(x, "x", torch.bfloat16, (ws.T, ws.H), dev)
    _require(topk_w, "topk_w", torch.float32, (ws.T, ws.k), dev)
    _require(dy, "dy", torch.bfloat16, (ws.T, ws.H), dev)
    _check_weights(ws, weights, "bwd")
    _check(mok_backward(ws.config.c(), _shape(ws.T, ws.H, ws.I, ws.E, ws.k), _ptr(schedule),
                        schedule.numel(), _ptr(ws.buffer), ws.buffer.numel(), _ptr(x), _ptr(topk_w), weights,
                        _ptr(fwd_ctx), fwd_ctx.numel(), _ptr(dy), _ptr(grads["dx"]),
                        _ptr(grads["dw_gate"]), _ptr(grads["dw_up"]), _ptr(grads["dw_down"]),
                        _ptr(grads["dtopk_w"]), _stream()), "mok_backward")
    return grads


def mxfp8_quantize(src, src_is_k_by_rows: bool):
    """src bf16 [B, rows, K] (or [B, K, rows] when src_is_k_by_rows). Returns
    (elems uint8 [B, rows, K], scales uint8 [B, rows, K/32])."""
    import torch
    if src.dim() != 3:
        raise ValueError(f"src: expected [B, rows, K] or [B, K, rows], got shape {tuple(src.shape)}")
    _require(src, "src", torch.bfloat16, tuple(src.shape))
    B = src.shape[0]
    rows, K = (src.shape[2], src.shape[1]) if src_is_k_by_rows else (src.shape[1], src.shape[2])
    elems = torch.empty((B, rows, K), dtype=torch.uint8, device=src.device)
    scales = torch.empty((B, rows, K // 32), dtype=torch.uint8, device=src.device)
    _check(mok_mxfp8_quantize(_ptr(src), B, rows, K, int(src_is_k_by_rows), _ptr(elems), _ptr(scales),
                              _stream()), "mok_mxfp8_quantize")
    return elems, scales


def route(logits, k: int):
    """logits fp32 [T, E] on the device. Returns (topk_ids int32 [T, k],
    topk_w fp32 [T, k]): the k largest logits per row and their softmax weights
    renormalised over the chosen k."""
    import torch
    T, E = logits.shape
    _require(logits, "logits", torch.float32, (T, E))
    ids = torch.empty((T, k), dtype=torch.int32, device=logits.device)
    w = torch.empty((T, k), dtype=torch.float32, device=logits.device)
    _check(mok_route(_ptr(logits), T, E, k, _ptr(ids), _ptr(w), _stream()), "mok_route")
    return ids, w


def route_backward(topk_ids, topk_w, dtopk_w, E: int):
    """Logit gradient fp32 [T, E] of route() for the upstream gradient dtopk_w [T, k]."""
    import torch
    T, k = topk_ids.shape
    _require(topk_ids, "topk_ids", torch.int32, (T, k))
    _require(topk_w, "topk_w", torch.float32, (T, k), topk_ids.device)
    _require(dtopk_w, "dtopk_w", torch.float32, (T, k), topk_ids.device)
    dl = torch.empty((T, E), dtype=torch.float32, device=topk_ids.device)
    _check(mok_route_backward(_ptr(topk_ids), _ptr(topk_w), _ptr(dtopk_w), T, E, k, _ptr(dl), _stream()),
           "mok_route_backward")
    return dl


# ----------------------------------------------------------------------------- around the routed experts

_STREAM_DTYPES = {torch.bfloat16: MOK_STREAM_BF16, torch.float32: MOK_STREAM_F32}
_BF16, _F32, _U8 = torch.bfloat16, torch.float32, torch.uint8


# These calls are short: for one decoded token the kernels take 3 to 25 us, so
# the host's share shows. The checks test the common case inline and leave the
# error's wording to _require; pointers go to ctypes as plain integers.

def _need(t, name, dtype, shape, device):
    try:
        if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.device == device:
            return
    except AttributeError:
        pass
    _require(t, name, dtype, shape, device)


# Argument structs by value (the library only reads them) and sizes by shape.
_norm_shape = functools.lru_cache(256)(mok_norm_shape)
_ffn_shape = functools.lru_cache(256)(mok_ffn_shape)


@functools.lru_cache(256)
def _norm_backward_bytes(T, H, sd) -> int:
    need = ctypes.c_size_t()
    _check(mok_add_rmsnorm_backward_size(mok_norm_shape(T, H, sd, 0.0, 0.0), ctypes.byref(need)),
           "mok_add_rmsnorm_backward_size")
    return need.value


def _addr(t):
    return None if t is None else t.data_ptr()


def _elsewhere(device) -> bool:
    """Whether device is not the current one: the kernels go to the device that
    holds the tensors, whatever device is current."""
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a GPU, got {device}")
    return _current_device() != device.index


# Without torch.cuda's own look at whether it is initialised, 0.5 us less: a tensor on the device says so.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
# torch.cuda.current_stream() builds a Stream object (1.9 us); the handle alone takes 0.1 us.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _stream_dtype(dtype, name):
    sd = _STREAM_DTYPES.get(dtype)
    if sd is None:
        raise ValueError(f"{name}: dtype {dtype}, expected torch.bfloat16 or torch.float32")
    return sd


def _rng_addr(p, rng, device):
    """rng: int64 [2] on the device, {seed, offset} as bit patterns; unused when p == 0."""
    if not 0.0 <= p < 1.0:
        raise ValueError(f"p: {p}, expected a value in [0, 1)")
    if p == 0.0:
        return None
    _need(rng, "rng", torch.int64, (2,), device)
    return rng.data_ptr()


def dropout(x, rng, p: float, residual=None, out=None):
    """residual + dropout(x) (mok_dropout). x: bf16, any shape; residual: bf16 or
    fp32 of that shape, or None; rng: int64 [2] on the device, {seed, offset}.
    Returns a tensor of residual's type (bf16 without one); ``out`` may be
    residual. A call draws (x.numel() + 3) // 4 counters from offset on."""
    shape, dev = x.shape, x.device
    like = x if residual is None else residual
    sd = _stream_dtype(like.dtype, "residual")
    _need(x, "x", _BF16, shape, dev)
    if residual is not None:
        _need(residual, "residual", residual.dtype, shape, dev)
    state = _rng_addr(p, rng, dev)
    if out is not None:
        _need(out, "out", like.dtype, shape, dev)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return dropout(x, rng, p, residual, out)
    if out is None:
        out = torch.empty_like(like)
    _check(_lib.mok_dropout(x.data_ptr(), _addr(residual), x.numel(), p, state, sd, out.data_ptr(),
                            _raw_stream(dev.index)), "mok_dropout")
    return out


def dropout_backward(dy, rng, p: float, dx=None):
    """Gradient of dropout() with respect to x, bf16 (mok_dropout_backward); p and
    rng as the forward had them. The residual's gradient is dy itself."""
    shape, dev = dy.shape, dy.device
    sd = _stream_dtype(dy.dtype, "dy")
    _need(dy, "dy", dy.dtype, shape, dev)
    state = _rng_addr(p, rng, dev)
    if dx is not None:
        _need(dx, "dx", _BF16, shape, dev)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return dropout_backward(dy, rng, p, dx)
    if dx is None:
        dx = torch.empty_like(dy, dtype=_BF16)
    _check(_lib.mok_dropout_backward(dy.data_ptr(), dy.numel(), p, state, sd, dx.data_ptr(), _raw_stream(dev.index)),
           "mok_dropout_backward")
    return dx


def add_rmsnorm(x, weight, eps: float, residual=None, p: float = 0.0, rng=None, stream_dtype=None, y: bool = True,
                mxfp8: bool = False, outs=None):
    """Residual addition (with dropout of x) and RMS norm (mok_add_rmsnorm).
    x: bf16 [T, H]; weight: bf16 [H]; residual: [T, H] in the stream's type or
    None. stream_dtype defaults to residual's type (bf16 without one). Returns a
    dict: sum [T, H] in the stream's type, rstd fp32 [T], y bf16 [T, H] (if
    ``y``), y_elems uint8 [T, H] and y_scales uint8 [T, H/32] (if ``mxfp8``).
    ``outs``: the same keys, caller-given; sum may be residual."""
    shape, dev = x.shape, x.device
    if len(shape) != 2:
        raise ValueError(f"x: shape {tuple(shape)}, expected [T, H]")
    T, H = shape
    dtype = stream_dtype or (_BF16 if residual is None else residual.dtype)
    sd = _stream_dtype(dtype, "stream_dtype")
    _need(x, "x", _BF16, shape, dev)
    _need(weight, "weight", _BF16, (H,), dev)
    if residual is not None:
        _need(residual, "residual", dtype, shape, dev)
    state = _rng_addr(p, rng, dev)
    if not y and not mxfp8:
        raise ValueError("y and mxfp8 are both off: nothing to write")
    if mxfp8 and H % 32:
        raise ValueError(f"x: H = {H}, MXFP8 rows need a multiple of 32")
    if outs is not None:
        _need(outs.get("sum"), "sum", dtype, shape, dev)
        _need(outs.get("rstd"), "rstd", _F32, (T,), dev)
        if y:
            _need(outs.get("y"), "y", _BF16, shape, dev)
        if mxfp8:
            _need(outs.get("y_elems"), "y_elems", _U8, shape, dev)
            _need(outs.get("y_scales"), "y_scales", _U8, (T, H // 32), dev)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return add_rmsnorm(x, weight, eps, residual, p, rng, stream_dtype, y, mxfp8, outs)
    if outs is None:
        r = dict(sum=torch.empty_like(x, dtype=dtype), rstd=x.new_empty((T,), dtype=_F32))
        if y:
            r["y"] = torch.empty_like(x)
        if mxfp8:
            r["y_elems"], r["y_scales"] = torch.empty_like(x, dtype=_U8), x.new_empty((T, H // 32), dtype=_U8)
    else:
        r = {n: outs[n] for n in ("sum", "rstd") + (("y",) if y else ()) + (("y_elems", "y_scales") if mxfp8 else ())}
    _check(_lib.mok_add_rmsnorm(ctypes.byref(_norm_shape(T, H, sd, eps, p)), x.data_ptr(), _addr(residual),
                                weight.data_ptr(), state, r["sum"].data_ptr(), r["y"].data_ptr() if y else None,
                                r["y_elems"].data_ptr() if mxfp8 else None,
                                r["y_scales"].data_ptr() if mxfp8 else None, r["rstd"].data_ptr(),
                                _raw_stream(dev.index)), "mok_add_rmsnorm")
    return r


def add_rmsnorm_backward(dy, sum, weight, rstd, dsum=None, p: float = 0.0, rng=None, grads=None, workspace=None):
    """Backward of add_rmsnorm() from its sum and rstd (mok_add_rmsnorm_backward).
    dy: bf16 [T, H]; dsum: [T, H] in sum's type, the gradient along the residual
    stream, or None. Returns a dict: dresidual [T, H] in sum's type, dx bf16
    [T, H], dweight fp32 [H]. ``grads``: the same keys, caller-given. Where both
    are bf16 and p == 0, dx equals dresidual: it is the same tensor then, unless
    ``grads`` holds a buffer of its own for it, which is written. ``workspace``:
    uint8, made here if None."""
    shape, dev, dtype = sum.shape, sum.device, sum.dtype
    if len(shape) != 2:
        raise ValueError(f"sum: shape {tuple(shape)}, expected [T, H]")
    T, H = shape
    sd = _stream_dtype(dtype, "sum")
    _need(sum, "sum", dtype, shape, dev)
    _need(dy, "dy", _BF16, shape, dev)
    _need(weight, "weight", _BF16, (H,), dev)
    _need(rstd, "rstd", _F32, (T,), dev)
    if dsum is not None:
        _need(dsum, "dsum", dtype, shape, dev)
    state = _rng_addr(p, rng, dev)
    separate = p > 0.0 or dtype is not _BF16
    if grads is not None:
        _need(grads.get("dresidual"), "dresidual", dtype, shape, dev)
        _need(grads.get("dweight"), "dweight", _F32, (H,), dev)
        if separate or grads.get("dx") is not None:
            _need(grads.get("dx"), "dx", _BF16, shape, dev)
            separate = separate or grads["dx"].data_ptr() != grads["dresidual"].data_ptr()
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return add_rmsnorm_backward(dy, sum, weight, rstd, dsum, p, rng, grads, workspace)
    need = _norm_backward_bytes(T, H, sd)
    if workspace is None:
        workspace = sum.new_empty((need,), dtype=_U8)
    else:
        _require_bytes(workspace, "workspace", need, dev)
        need = workspace.numel()
    if grads is None:
        g = dict(dresidual=torch.empty_like(sum), dweight=torch.empty_like(weight, dtype=_F32))
        if separate:
            g["dx"] = torch.empty_like(dy)
    else:
        g = {n: grads[n] for n in ("dresidual", "dweight") + (("dx",) if separate else ())}
    _check(_lib.mok_add_rmsnorm_backward(ctypes.byref(_norm_shape(T, H, sd, 0.0, p)), workspace.data_ptr(), need,
                                         dy.data_ptr(), sum.data_ptr(), weight.data_ptr(), rstd.data_ptr(),
                                         _addr(dsum), state, g["dresidual"].data_ptr(),
                                         g["dx"].data_ptr() if separate else None, g["dweight"].data_ptr(),
                                         _raw_stream(dev.index)), "mok_add_rmsnorm_backward")
    if not separate:
        g["dx"] = g["dresidual"]
    return g


@dataclasses.dataclass
class FfnWorkspace:
    """Caller-owned scratch of the feed-forward block for up to T rows (made once, reused)."""
    precision: int
    T: int
    H: int
    I: int
    buffer: "object"        # torch.uint8 tensor


def get_ffn_workspace(precision: int = MOK_BF16, *, device, num_tokens: int, hidden_size: int,
                      intermediate_size: int) -> FfnWorkspace:
    need = ctypes.c_size_t()
    _check(mok_ffn_query_size(mok_ffn_shape(num_tokens, hidden_size, intermediate_size, precision),
                              ctypes.byref(need)), "mok_ffn_query_size")
    buf = torch.empty(need.value, dtype=torch.uint8, device=device)
    return FfnWorkspace(precision, num_tokens, hidden_size, intermediate_size, buf)


def _check_ffn_weights(ws: FfnWorkspace, weights: mok_weights, orientation: str):
    """Shapes, dtypes and devices of the tensors a weight struct refers to: one
    expert's, with or without a leading dimension of 1."""
    tensors = getattr(weights, "_tensors", None)
    if tensors is None:          # a hand-made struct: nothing to check against
        return
    dev, H, I = ws.buffer.device, ws.H, ws.I
    kind = getattr(weights, "_kind", "")

    def one(t, name, dtype, shape):
        _need(t, name, dtype, (1,) + shape if t.dim() == 3 else shape, dev)

    if ws.precision == MOK_BF16:
        if not kind.startswith("bf16"):
            raise ValueError("BF16 mode needs bf16 weights (weights_bf16)")
        g, u, d = tensors
        one(g, "w_gate", _BF16, (H, I))
        one(u, "w_up", _BF16, (H, I))
        one(d, "w_down", _BF16, (I, H))
        return
    if not kind.startswith("mxfp8"):
        raise ValueError("MXFP8 mode needs quantized weights (MXFP8Weights)")
    if ":" in kind and kind.split(":")[1] != orientation:
        raise ValueError(f"MXFP8 weights quantized for {kind.split(':')[1]}, used in {orientation}")
    shapes = ((I, H), (I, H), (H, I)) if orientation == "fwd" else ((H, I), (H, I), (I, H))
    for (el, sc), n, sh in zip(tensors, ("gate", "up", "down"), shapes):
        one(el, n + " elements", _U8, sh)
        one(sc, n + " scales", _U8, (sh[0], sh[1] // 32))


def _ffn_rows(ws: FfnWorkspace, t, name):
    if t.dim() != 2 or t.shape[0] > ws.T:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected [T, {ws.H}] with T <= {ws.T}")
    return t.shape[0]


def ffn_forward(ws: FfnWorkspace, x, weights: mok_weights, addend=None, out=None, h=None, save_h: bool = True):
    """Dense gated feed-forward block (mok_ffn_forward): out = addend +
    (silu(x W_gate) * (x W_up)) W_down. x: bf16 [T, H] (T up to ws.T), or in
    MXFP8 the pair (elems uint8 [T, H], scales uint8 [T, H/32]) that
    add_rmsnorm(mxfp8=True) gives, or mxfp8_quantize of x[None] without its
    leading dimension. addend: bf16 [T, H] or None;
    ``out`` may be addend. Returns (out bf16 [T, H], h bf16 [T, 2I] for the
    backward, or None with save_h=False and no ``h``)."""
    buf, H, I = ws.buffer, ws.H, ws.I
    dev = buf.device
    if ws.precision == MOK_BF16:
        T = _ffn_rows(ws, x, "x")
        _need(x, "x", _BF16, (T, H), dev)
        rows, elems, scales = x.data_ptr(), None, None
    else:
        if not isinstance(x, (tuple, list)) or len(x) != 2:
            raise ValueError("x: MXFP8 mode takes (elems, scales)")
        el, sc = x
        T = _ffn_rows(ws, el, "x elements")
        _need(el, "x elements", _U8, (T, H), dev)
        _need(sc, "x scales", _U8, (T, H // 32), dev)
        rows, elems, scales = None, el.data_ptr(), sc.data_ptr()
    _check_ffn_weights(ws, weights, "fwd")
    if addend is not None:
        _need(addend, "addend", _BF16, (T, H), dev)
    if out is not None:
        _need(out, "out", _BF16, (T, H), dev)
    if h is not None:
        _need(h, "h", _BF16, (T, 2 * I), dev)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return ffn_forward(ws, x, weights, addend, out, h, save_h)
    if out is None:
        out = buf.new_empty((T, H), dtype=_BF16)
    if h is None and save_h:
        h = buf.new_empty((T, 2 * I), dtype=_BF16)
    _check(_lib.mok_ffn_forward(ctypes.byref(_ffn_shape(T, H, I, ws.precision)), buf.data_ptr(), buf.numel(), rows,
                                elems, scales, ctypes.byref(weights), _addr(addend), out.data_ptr(), _addr(h),
                                _raw_stream(dev.index)), "mok_ffn_forward")
    return out, h


def ffn_backward(ws: FfnWorkspace, x, weights: mok_weights, h, dy, addend=None, grads=None):
    """Backward of ffn_forward() (mok_ffn_backward). x: bf16 [T, H] in either
    precision; weights: in MXFP8 the backward's orientation; addend: bf16 [T, H]
    added to dx, or None. Returns dict(dx, dw_gate, dw_up, dw_down), bf16;
    ``grads``: the same keys, caller-given (dx may be addend)."""
    buf, H, I = ws.buffer, ws.H, ws.I
    dev = buf.device
    T = _ffn_rows(ws, x, "x")
    _need(x, "x", _BF16, (T, H), dev)
    _need(h, "h", _BF16, (T, 2 * I), dev)
    _need(dy, "dy", _BF16, (T, H), dev)
    if addend is not None:
        _need(addend, "addend", _BF16, (T, H), dev)
    _check_ffn_weights(ws, weights, "bwd")
    shapes = dict(dx=(T, H), dw_gate=(H, I), dw_up=(H, I), dw_down=(I, H))
    if grads is not None:
        for n, sh in shapes.items():
            _need(grads.get(n), n, _BF16, sh, dev)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return ffn_backward(ws, x, weights, h, dy, addend, grads)
    g = {n: buf.new_empty(sh, dtype=_BF16) if grads is None else grads[n] for n, sh in shapes.items()}
    _check(_lib.mok_ffn_backward(ctypes.byref(_ffn_shape(T, H, I, ws.precision)), buf.data_ptr(), buf.numel(),
                                 x.data_ptr(), ctypes.byref(weights), h.data_ptr(), dy.data_ptr(), _addr(addend),
                                 g["dx"].data_ptr(), g["dw_gate"].data_ptr(), g["dw_up"].data_ptr(),
                                 g["dw_down"].data_ptr(), _raw_stream(dev.index)), "mok_ffn_backward")
    return g


# ----------------------------------------------------------------------------- the routed experts taken apart

_I32 = torch.int32


@functools.lru_cache(256)
def _rows_shape(T, rows, k, E, H, dtype):
    return ctypes.byref(mok_rows_shape(T, rows, k, E, H, dtype))


@functools.lru_cache(256)
def _sort_sizes(T, k, E, align):
    shape, rows, need = mok_sort_shape(T, k, E, align), ctypes.c_int64(), ctypes.c_size_t()
    _check(mok_sort_tokens_size(shape, ctypes.byref(rows), ctypes.byref(need)), "mok_sort_tokens_size")
    return ctypes.byref(shape), rows.value, need.value


@functools.lru_cache(256)
def _fp8_plan(wgrad, M, N, K, E, dtype):
    """The argument struct and the workspace bytes of a product."""
    shape, need = mok_fp8_shape(M, N, K, E, dtype), ctypes.c_size_t()
    size, name = (mok_fp8_wgrad_size, "mok_fp8_wgrad_size") if wgrad else (mok_fp8_matmul_size, "mok_fp8_matmul_size")
    _check(size(shape, ctypes.byref(need)), name)
    return ctypes.byref(shape), need.value


def _given_workspace(workspace, need, like):
    if workspace is None and need == 0:
        return None
    if workspace is None:
        return like.new_empty((need,), dtype=_U8)
    _require_bytes(workspace, "workspace", need, like.device)
    return workspace


def sort_rows(num_tokens: int, topk: int, num_experts: int, align: int = 1) -> int:
    """Most rows that a sort of these sizes fills (mok_sort_tokens_size)."""
    return _sort_sizes(num_tokens, topk, num_experts, align)[1]


def sort_tokens(topk_ids, num_experts: int, align: int = 1, outs=None, workspace=None):
    """Sort of token slots by expert (mok_sort_tokens). topk_ids: int32 [T, k]; an
    id outside [0, num_experts) names no expert here. Every expert's run of rows
    is rounded up to a multiple of ``align``. Returns a dict of int32 tensors:
    offsets [E + 1], slots [T, k] (each slot's row, or -1) and row_slots [rows]
    (each row's slot t * k + j, or -1), rows as sort_rows() gives. ``outs``: the
    same keys, caller-given; ``workspace``: uint8, made here if None."""
    shape, dev = topk_ids.shape, topk_ids.device
    if len(shape) != 2:
        raise ValueError(f"topk_ids: shape {tuple(shape)}, expected [T, k]")
    T, k = shape
    _need(topk_ids, "topk_ids", _I32, shape, dev)
    c, rows, need = _sort_sizes(T, k, num_experts, align)
    if outs is not None:
        _need(outs.get("offsets"), "offsets", _I32, (num_experts + 1,), dev)
        _need(outs.get("slots"), "slots", _I32, shape, dev)
        _need(outs.get("row_slots"), "row_slots", _I32, (rows,), dev)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return sort_tokens(topk_ids, num_experts, align, outs, workspace)
    ws = _given_workspace(workspace, need, topk_ids)
    if outs is None:
        r = dict(offsets=topk_ids.new_empty((num_experts + 1,)), slots=torch.empty_like(topk_ids),
                 row_slots=topk_ids.new_empty((rows,)))
    else:
        r = {n: outs[n] for n in ("offsets", "slots", "row_slots")}
    _check(_lib.mok_sort_tokens(c, _addr(ws), need, topk_ids.data_ptr(),
                                r["offsets"].data_ptr(), r["slots"].data_ptr(), r["row_slots"].data_ptr(),
                                _raw_stream(dev.index)), "mok_sort_tokens")
    return r


def _sort_of(sort, device):
    """(T, k, rows, E) of a sort_tokens() dict, its tensors checked."""
    slots, row_slots, offsets = sort["slots"], sort["row_slots"], sort["offsets"]
    shape = slots.shape
    if len(shape) != 2 or row_slots.dim() != 1 or offsets.dim() != 1 or offsets.numel() < 2:
        raise ValueError("sort: expected slots [T, k], row_slots [rows] and offsets [E + 1]")
    if not (slots.dtype is _I32 and row_slots.dtype is _I32 and offsets.dtype is _I32 and slots.is_contiguous()
            and row_slots.is_contiguous() and offsets.is_contiguous() and slots.device == device
            and row_slots.device == device and offsets.device == device):
        for t, name in ((slots, "slots"), (row_slots, "row_slots"), (offsets, "offsets")):
            _require(t, name, _I32, t.shape, device)
    return shape[0], shape[1], row_slots.numel(), offsets.numel() - 1


def _rows_of(t, name, n):
    """H of a tensor of n rows, checked."""
    shape = t.shape
    if len(shape) != 2 or shape[0] != n:
        raise ValueError(f"{name}: shape {tuple(shape)}, expected [{n}, H]")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return shape[1]


def permute(x, sort, rows: bool = True, fp8: bool = False, outs=None):
    """Token rows into their experts' order (mok_permute). x: bf16 or fp32 [T, H];
    sort: what sort_tokens() returned. Returns a dict: rows [rows, H] in x's type
    (if ``rows``), elems uint8 [rows, H] and scales fp32 [ceil(H/128), rows] (if
    ``fp8``: the rows quantized in blocks of 128). Rows behind the last expert's
    run are not written. ``outs``: the same keys, caller-given."""
    dev = x.device
    sd = _stream_dtype(x.dtype, "x")
    T, k, n, E = _sort_of(sort, dev)
    H = _rows_of(x, "x", T)
    if not rows and not fp8:
        raise ValueError("rows and fp8 are both off: nothing to write")
    if H % 8 or (fp8 and H % 16):
        raise ValueError(f"x: H = {H}, expected a multiple of {16 if fp8 else 8}")
    kb = (H + 127) // 128
    if outs is not None:
        if rows:
            _need(outs.get("rows"), "rows", x.dtype, (n, H), dev)
        if fp8:
            _need(outs.get("elems"), "elems", _U8, (n, H), dev)
            _need(outs.get("scales"), "scales", _F32, (kb, n), dev)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return permute(x, sort, rows, fp8, outs)
    if outs is None:
        r = dict(rows=x.new_empty((n, H))) if rows else {}
        if fp8:
            r["elems"], r["scales"] = x.new_empty((n, H), dtype=_U8), x.new_empty((kb, n), dtype=_F32)
    else:
        r = {name: outs[name] for name in (("rows",) if rows else ()) + (("elems", "scales") if fp8 else ())}
    _check(_lib.mok_permute(_rows_shape(T, n, k, E, H, sd), x.data_ptr(), sort["offsets"].data_ptr(),
                            sort["slots"].data_ptr(), sort["row_slots"].data_ptr(), _addr(r.get("rows")),
                            _addr(r.get("elems")), _addr(r.get("scales")), _raw_stream(dev.index)), "mok_permute")
    return r


def permute_backward(drows, sort, dx=None):
    """Gradient of permute() with respect to x (mok_permute_backward): the sum of
    each token's rows. drows: bf16 or fp32 [rows, H]. Returns [T, H] in its type."""
    dev = drows.device
    sd = _stream_dtype(drows.dtype, "drows")
    T, k, n, E = _sort_of(sort, dev)
    H = _rows_of(drows, "drows", n)
    if dx is not None:
        _need(dx, "dx", drows.dtype, (T, H), dev)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return permute_backward(drows, sort, dx)
    if dx is None:
        dx = drows.new_empty((T, H))
    _check(_lib.mok_permute_backward(_rows_shape(T, n, k, E, H, sd), drows.data_ptr(),
                                     sort["slots"].data_ptr(), dx.data_ptr(), _raw_stream(dev.index)),
           "mok_permute_backward")
    return dx


def unpermute(y, sort, w=None, addend=None, out=None):
    """The experts' rows back in token order (mok_unpermute): out[t] = addend[t] +
    sum over j of w[t, j] * y[slots[t, j]]. y: bf16 or fp32 [rows, H]; w: fp32
    [T, k] or None (ones); addend: [T, H] in y's type or None (its gradient is
    out's). ``out`` may be addend."""
    dev = y.device
    sd = _stream_dtype(y.dtype, "y")
    T, k, n, E = _sort_of(sort, dev)
    H = _rows_of(y, "y", n)
    if w is not None:
        _need(w, "w", _F32, (T, k), dev)
    if addend is not None:
        _need(addend, "addend", y.dtype, (T, H), dev)
    if out is not None:
        _need(out, "out", y.dtype, (T, H), dev)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return unpermute(y, sort, w, addend, out)
    if out is None:
        out = y.new_empty((T, H))
    _check(_lib.mok_unpermute(_rows_shape(T, n, k, E, H, sd), y.data_ptr(), sort["slots"].data_ptr(),
                              _addr(w), _addr(addend), out.data_ptr(), _raw_stream(dev.index)), "mok_unpermute")
    return out


def unpermute_backward(dout, y, sort, w, grads=None):
    """Gradient of unpermute() with weights (mok_unpermute_backward). dout: [T, H],
    y: [rows, H] in the same type, as the forward read it; w: fp32 [T, k]. Returns
    dict(dy [rows, H], dw fp32 [T, k]); rows behind the last expert's run are not
    written. ``grads``: the same keys, caller-given (dy may be y). Without weights
    the gradient is permute(dout, sort)."""
    dev = y.device
    sd = _stream_dtype(y.dtype, "y")
    T, k, n, E = _sort_of(sort, dev)
    H = _rows_of(y, "y", n)
    _need(dout, "dout", y.dtype, (T, H), dev)
    _need(w, "w", _F32, (T, k), dev)
    if grads is not None:
        _need(grads.get("dy"), "dy", y.dtype, (n, H), dev)
        _need(grads.get("dw"), "dw", _F32, (T, k), dev)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return unpermute_backward(dout, y, sort, w, grads)
    g = dict(dy=torch.empty_like(y), dw=torch.empty_like(w)) if grads is None else dict(dy=grads["dy"], dw=grads["dw"])
    _check(_lib.mok_unpermute_backward(_rows_shape(T, n, k, E, H, sd), dout.data_ptr(), y.data_ptr(),
                                       sort["offsets"].data_ptr(), sort["slots"].data_ptr(),
                                       sort["row_slots"].data_ptr(), w.data_ptr(), g["dy"].data_ptr(),
                                       g["dw"].data_ptr(), _raw_stream(dev.index)), "mok_unpermute_backward")
    return g


def fp8_quantize(src, src_is_k_by_rows: bool = False, tile: bool = False, glu: bool = False, outs=None):
    """Quantization to E4M3 with one fp32 scale per block of 128 (mok_fp8_quantize).
    src: bf16 or fp32 [B, rows, K], or [B, K, rows] when src_is_k_by_rows
    (quantizes the transpose). A block is 128 values along K, or with ``tile`` 128
    rows x 128 values. With ``glu`` (bf16, no tile) src is [.., 2K] (or [B, K,
    2 * rows]) and silu(g) * u of its halves is quantized. Returns (elems uint8
    [B, rows, K], scales fp32 [B, ceil(K/128), rows], or with ``tile``
    [B, ceil(rows/128), ceil(K/128)]); ``outs``: such a pair, caller-given."""
    dev = src.device
    if src.dim() != 3:
        raise ValueError(f"src: expected [B, rows, K] or [B, K, rows], got shape {tuple(src.shape)}")
    sd = _stream_dtype(src.dtype, "src")
    if not src.is_contiguous():
        raise ValueError("src: must be contiguous")
    B, middle, last = src.shape
    if glu:
        if tile or sd != MOK_STREAM_BF16:
            raise ValueError("glu takes bf16 rows and no tile")
        if last % 2:
            raise ValueError(f"src: last dimension {last}, expected two halves")
        last //= 2
    rows, K = (last, middle) if src_is_k_by_rows else (middle, last)
    if K % 16 or (src_is_k_by_rows and rows % 8):
        raise ValueError(f"src: K = {K}, rows = {rows}: K must be a multiple of 16"
                         + (" and rows of 8" if src_is_k_by_rows else ""))
    kb = (K + 127) // 128
    sshape = (B, (rows + 127) // 128, kb) if tile else (B, kb, rows)
    if outs is not None:
        if not isinstance(outs, (tuple, list)) or len(outs) != 2:
            raise ValueError("outs: expected (elems, scales)")
        _need(outs[0], "elems", _U8, (B, rows, K), dev)
        _need(outs[1], "scales", _F32, sshape, dev)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return fp8_quantize(src, src_is_k_by_rows, tile, glu, outs)
    if outs is None:
        outs = src.new_empty((B, rows, K), dtype=_U8), src.new_empty(sshape, dtype=_F32)
    elems, scales = outs
    flags = (MOK_FP8_TURNED if src_is_k_by_rows else 0) | (MOK_FP8_TILE if tile else 0) | (MOK_FP8_GLU if glu else 0)
    _check(_lib.mok_fp8_quantize(src.data_ptr(), sd, B, rows, K, flags, elems.data_ptr(), scales.data_ptr(),
                                 _raw_stream(dev.index)), "mok_fp8_quantize")
    return elems, scales


def glu_backward(da, h, dh=None):
    """Gradient of a = silu(g) * u with respect to h = [g | u] (mok_glu_backward).
    da: bf16 [T, I], h: bf16 [T, 2I]. Returns bf16 [T, 2I]; ``dh`` may be h."""
    dev = da.device
    if da.dim() != 2 or da.shape[1] % 8:
        raise ValueError(f"da: shape {tuple(da.shape)}, expected [T, I] with I a multiple of 8")
    T, I = da.shape
    _need(da, "da", _BF16, (T, I), dev)
    _need(h, "h", _BF16, (T, 2 * I), dev)
    if dh is not None:
        _need(dh, "dh", _BF16, (T, 2 * I), dev)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return glu_backward(da, h, dh)
    if dh is None:
        dh = torch.empty_like(h)
    _check(_lib.mok_glu_backward(da.data_ptr(), h.data_ptr(), T, I, dh.data_ptr(), _raw_stream(dev.index)),
           "mok_glu_backward")
    return dh


def _pair(t, name):
    if not isinstance(t, (tuple, list)) or len(t) != 2:
        raise ValueError(f"{name}: expected (elems, scales)")
    return t


def _row_codes(t, name, device=None):
    """(elems, scales, rows, K) of rows quantized in blocks of 128, with or without a leading dimension of 1."""
    el, sc = _pair(t, name)
    if el.dim() == 3 and el.shape[0] == 1 and sc.dim() == 3:
        el, sc = el[0], sc[0]
    shape = el.shape
    if len(shape) != 2:
        raise ValueError(f"{name} elems: shape {tuple(shape)}, expected [rows, K]")
    rows, K = shape
    dev = el.device if device is None else device
    if not (el.dtype is _U8 and el.is_contiguous() and (device is None or el.device == dev)):
        _require(el, name + " elems", _U8, shape, dev)
    _need(sc, name + " scales", _F32, ((K + 127) // 128, rows), dev)
    return el, sc, rows, K


def _experts(offsets, device):
    if offsets is None:
        return 0
    if offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError(f"offsets: shape {tuple(offsets.shape)}, expected [E + 1]")
    _need(offsets, "offsets", _I32, offsets.shape, device)
    return offsets.shape[0] - 1


def fp8_matmul(a, b, offsets=None, out_dtype=torch.bfloat16, out=None, workspace=None):
    """a @ b^T on operands in blocks of 128 (mok_fp8_matmul). a: (elems uint8
    [M, K], scales fp32 [ceil(K/128), M]), rows of fp8_quantize or permute; b:
    (elems uint8 [N, K], scales fp32 [ceil(N/128), ceil(K/128)]), tiles. With
    ``offsets`` (int32 [E + 1] on the device, as sort_tokens returns them) b has a
    leading dimension E and rows [offsets[e], offsets[e + 1]) meet b[e]; rows of
    no expert are not written. Returns bf16 or fp32 [M, N]; ``out``: caller-given,
    in the type it has. N and K are multiples of 16."""
    el, sc, M, K = _row_codes(a, "a")
    dev = el.device
    E = _experts(offsets, dev)
    bel, bsc = _pair(b, "b")
    if E == 0 and bel.dim() == 3 and bel.shape[0] == 1 and bsc.dim() == 3:
        bel, bsc = bel[0], bsc[0]
    if bel.dim() != (3 if E else 2):
        raise ValueError(f"b elems: shape {tuple(bel.shape)}, expected " + ("[E, N, K]" if E else "[N, K]"))
    N = bel.shape[-2]
    lead = (E,) if E else ()
    _need(bel, "b elems", _U8, lead + (N, K), dev)
    _need(bsc, "b scales", _F32, lead + ((N + 127) // 128, (K + 127) // 128), dev)
    if N % 16 or K % 16:
        raise ValueError(f"N = {N}, K = {K}: expected multiples of 16")
    if out is not None:
        out_dtype = out.dtype
        _need(out, "out", out_dtype, (M, N), dev)
    sd = _stream_dtype(out_dtype, "out")
    c, need = _fp8_plan(False, M, N, K, E, sd)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return fp8_matmul(a, b, offsets, out_dtype, out, workspace)
    ws = _given_workspace(workspace, need, el)
    if out is None:
        out = el.new_empty((M, N), dtype=out_dtype)
    _check(_lib.mok_fp8_matmul(c, _addr(ws), need, el.data_ptr(),
                               sc.data_ptr(), bel.data_ptr(), bsc.data_ptr(), _addr(offsets), out.data_ptr(),
                               _raw_stream(dev.index)), "mok_fp8_matmul")
    return out


def fp8_wgrad(dy, x, offsets=None, out_dtype=torch.bfloat16, addend=None, out=None, workspace=None):
    """Weight gradient addend + dy^T x over the rows of each expert (mok_fp8_wgrad).
    dy: (elems uint8 [N, R], scales fp32 [ceil(R/128), N]), x: (elems uint8 [K, R],
    scales fp32 [ceil(R/128), K]), both from fp8_quantize(.., src_is_k_by_rows=True)
    of the R rows. ``offsets``: int32 [E + 1] whose runs start at multiples of 128
    (sort_tokens with align=128; one that starts elsewhere gives NaN) and end at
    any row, or None for one product. Returns [E, N, K] or [N, K] in bf16 or fp32;
    ``addend`` and ``out`` have that shape, and ``out`` may be addend. N, K and R
    are multiples of 16."""
    el, sc, N, R = _row_codes(dy, "dy")
    dev = el.device
    xel, xsc, K, R2 = _row_codes(x, "x", dev)
    if R2 != R:
        raise ValueError(f"x elems: {R2} rows along the contraction, dy has {R}")
    if N % 16 or K % 16 or R % 16:
        raise ValueError(f"N = {N}, K = {K}, R = {R}: expected multiples of 16")
    E = _experts(offsets, dev)
    shape = ((E,) if E else ()) + (N, K)
    if out is not None:
        out_dtype = out.dtype
        _need(out, "out", out_dtype, shape, dev)
    sd = _stream_dtype(out_dtype, "out")
    if addend is not None:
        _need(addend, "addend", out_dtype, shape, dev)
    c, need = _fp8_plan(True, R, N, K, E, sd)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return fp8_wgrad(dy, x, offsets, out_dtype, addend, out, workspace)
    ws = _given_workspace(workspace, need, el)
    if out is None:
        out = el.new_empty(shape, dtype=out_dtype)
    _check(_lib.mok_fp8_wgrad(c, _addr(ws), need, el.data_ptr(),
                              sc.data_ptr(), xel.data_ptr(), xsc.data_ptr(), _addr(offsets), _addr(addend),
                              out.data_ptr(), _raw_stream(dev.index)), "mok_fp8_wgrad")
    return out


def read_schedule(schedule, layout: mok_schedule_layout, E: int):
    """Copy the schedule table's fields to host numpy arrays (synchronises)."""
    import numpy as np
    host = schedule.cpu().numpy()

    def i32(off, n):
        return host[off: off + 4 * n].view(np.int32).copy()
    R, NM, G = layout.R, layout.NM, layout.G
    n_seg = int(i32(layout.n_seg, 1)[0])
    return dict(status=int(host[layout.status: layout.status + 4].view(np.uint32)[0]), n_seg=n_seg,
                counts=i32(layout.counts, E), offsets=i32(layout.offsets, E + 1),
                mcounts=i32(layout.mcounts, NM * E).reshape(NM, E),
                moffsets=i32(layout.moffsets, NM * (E + 1)).reshape(NM, E + 1),
                perm=i32(layout.perm, R), inv=i32(layout.inv, R), canon=i32(layout.canon, R),
                mb_start=i32(layout.mb_start, G + 1),
                segments=i32(layout.segments, 4 * min(n_seg, layout.cap)).reshape(-1, 4))
