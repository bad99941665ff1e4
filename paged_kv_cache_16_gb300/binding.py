"""ctypes binding of libpa.so: argument marshalling only.

Every function here forwards to the C ABI declared in ``include/pa.h`` with
the same name; device tensors are passed as raw pointers (``data_ptr()``)
and streams as ``cudaStream_t`` handles.  No step of the computation runs in
Python: if the compiled library is missing, loading fails with an error.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import numpy as np

from . import build as _build

PA_OK = 0
PA_ERR_INVALID_ARGUMENT = 1
PA_ERR_UNSUPPORTED = 2
PA_ERR_CUDA = 3
PA_ERR_DEVICE_CHECK = 4
PA_ERR_WORKSPACE_TOO_SMALL = 5
PA_ERR_CAPACITY = 6

PA_KV_BF16 = 0
PA_KV_FP8_E4M3 = 1
PA_KV_FP8_E4M3_BLOCK = 2
PA_KV_INT8_BLOCK = 3

PA_ROPE_HALF = 0
PA_ROPE_INTERLEAVED = 1
PA_ROPE_SCALE_NONE = 0
PA_ROPE_SCALE_LINEAR = 1
PA_ROPE_SCALE_WAVELENGTH = 2
PA_ROPE_SCALE_YARN = 3
PA_ROPE_AXES_SHARED = 0
PA_ROPE_AXES_OWN = 1

PA_DEVERR_SLOT_RANGE = 0x1
PA_DEVERR_BLOCK_RANGE = 0x2
PA_DEVERR_TIMEOUT = 0x4

# symbols include/pa.h declares (checked by the CPU tests)
EXPORTED = ("pa_plan", "pa_plan_destroy", "pa_plan_get_info", "pa_slot_mapping", "pa_write_kv",
            "pa_attention", "pa_check_device_errors", "pa_plan_enable_timing",
            "pa_plan_kernel_times", "pa_status_string", "pa_attention_no_alloc", "pa_write_kv_fp8",
            "pa_plan_fixed", "pa_upload_metadata", "pa_attention_launch", "pa_zero_blocks",
            "pa_attention_with_kv_update", "pa_attention_with_kv_update_launch", "pa_plan_metadata_bytes",
            "pa_plan_copy_metadata", "pa_upload_metadata_from", "pa_graph_create", "pa_graph_step",
            "pa_graph_turn", "pa_graph_wait", "pa_graph_workspace", "pa_graph_slot_mapping", "pa_graph_destroy",
            "pa_attention_with_kv_update_launch_staged", "pa_rope_create", "pa_rope_destroy", "pa_rope_frequencies",
            "pa_rotary", "pa_append_kv", "pa_attention_scaled", "pa_attention_scaled_launch", "pa_plan_window",
            "pa_rope_create_axes", "pa_rotary_axes", "pa_append_kv_axes")


class PaError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} ({status})")
        self.status = status


class BatchDesc(ctypes.Structure):
    _fields_ = [
        ("num_reqs", ctypes.c_int32),
        ("num_heads_q", ctypes.c_int32),
        ("num_heads_kv", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("block_size", ctypes.c_int32),
        ("num_blocks", ctypes.c_int32),
        ("max_blocks_per_req", ctypes.c_int32),
        ("query_start_loc", ctypes.c_void_p),      # const int32_t * (host)
        ("seq_lens", ctypes.c_void_p),
        ("num_computed_tokens", ctypes.c_void_p),
        ("block_table_host", ctypes.c_void_p),
        ("num_common_prefix_blocks", ctypes.c_int32),
        ("softmax_scale", ctypes.c_float),
        ("num_sms", ctypes.c_int32),
        ("kv_cache_dtype", ctypes.c_int32),
        ("k_scale", ctypes.c_float),
        ("v_scale", ctypes.c_float),
    ]


class PlanInfo(ctypes.Structure):
    _fields_ = [
        ("num_tokens", ctypes.c_int32),
        ("num_decode_rows", ctypes.c_int32),
        ("num_extend_rows", ctypes.c_int32),
        ("num_decode_ctas", ctypes.c_int32),
        ("num_decode_items", ctypes.c_int32),
        ("num_extend_tiles", ctypes.c_int32),
        ("num_prefix_tiles", ctypes.c_int32),
        ("num_partial_slots", ctypes.c_int32),
        ("num_merge_rows", ctypes.c_int32),
        ("kernels_per_call", ctypes.c_int32),
        ("num_dequant_blocks", ctypes.c_int32),
        ("decode_kv_bytes", ctypes.c_int64),
        ("prefix_kv_bytes", ctypes.c_int64),
        ("extend_flops", ctypes.c_double),
        ("prefix_flops", ctypes.c_double),
        ("num_small_q_rows", ctypes.c_int32),
        ("num_extend_ctas", ctypes.c_int32),
        ("side_by_side", ctypes.c_int32),
    ]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


_LIB = None


class FixedShape(ctypes.Structure):
    _fields_ = [
        ("max_tokens", ctypes.c_int32),
        ("max_reqs", ctypes.c_int32),
        ("max_extend_tiles", ctypes.c_int32),
        ("max_dequant_blocks", ctypes.c_int32),
        ("max_partial_slots", ctypes.c_int32),
        ("decode_prefix_tokens", ctypes.c_int32),
    ]


class GraphBuffers(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p),
        ("key", ctypes.c_void_p),
        ("value", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
        ("query_start_loc", ctypes.c_void_p),
        ("num_computed", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p),
        ("key_cache", ctypes.c_void_p),
        ("value_cache", ctypes.c_void_p),
        ("fused", ctypes.c_int32),
        ("host_in", ctypes.c_void_p * 2),
        ("device_in", ctypes.c_void_p),
        ("in_bytes", ctypes.c_size_t),
        ("host_out", ctypes.c_void_p * 2),
        ("out_bytes", ctypes.c_size_t),
    ]


class RopeDesc(ctypes.Structure):
    _fields_ = [
        ("rotary_dim", ctypes.c_int32),
        ("layout", ctypes.c_int32),
        ("scaling", ctypes.c_int32),
        ("original_max_position", ctypes.c_int32),
        ("base", ctypes.c_double),
        ("factor", ctypes.c_double),
        ("low", ctypes.c_double),
        ("high", ctypes.c_double),
        ("attention_factor", ctypes.c_double),
    ]


class RopeAxesDesc(ctypes.Structure):
    _fields_ = [
        ("num_axes", ctypes.c_int32),
        ("frequencies", ctypes.c_int32),
        ("axis_of_pair", ctypes.c_void_p),         # const int32_t * (host)
    ]


class WindowDesc(ctypes.Structure):
    _fields_ = [
        ("window", ctypes.c_int32),
        ("sink_tokens", ctypes.c_int32),
    ]


class AppendArgs(ctypes.Structure):
    _fields_ = [
        ("num_reqs", ctypes.c_int32),
        ("num_tokens", ctypes.c_int32),
        ("num_heads_q", ctypes.c_int32),
        ("num_heads_kv", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("block_size", ctypes.c_int32),
        ("num_blocks", ctypes.c_int32),
        ("max_blocks_per_req", ctypes.c_int32),
        ("kv_cache_dtype", ctypes.c_int32),
        ("k_scale", ctypes.c_float),
        ("v_scale", ctypes.c_float),
        ("query_start_loc", ctypes.c_void_p),
        ("num_computed_tokens", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p),
        ("key", ctypes.c_void_p),
        ("value", ctypes.c_void_p),
        ("key_stride", ctypes.c_int64),
        ("value_stride", ctypes.c_int64),
        ("q", ctypes.c_void_p),
        ("q_out", ctypes.c_void_p),
        ("q_stride", ctypes.c_int64),
        ("q_out_stride", ctypes.c_int64),
        ("key_cache", ctypes.c_void_p),
        ("value_cache", ctypes.c_void_p),
        ("key_scales", ctypes.c_void_p),
        ("value_scales", ctypes.c_void_p),
        ("device_error_word", ctypes.c_void_p),
    ]


def library_path() -> str:
    return _build.LIBRARY


def load(path: str | None = None, build_if_missing: bool = False) -> ctypes.CDLL:
    """Load libpa.so (optionally building it first)."""
    global _LIB
    if _LIB is not None and path is None:
        return _LIB
    p = path or _build.LIBRARY
    if not os.path.exists(p):
        if build_if_missing:
            p = _build.build()
        else:
            raise RuntimeError(f"libpa.so not built ({p}); run paged_kv_cache_16_gb300.build.build()")
    lib = ctypes.CDLL(p)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    i32p = ctypes.POINTER(ctypes.c_int32)
    lib.pa_status_string.restype = ctypes.c_char_p
    lib.pa_status_string.argtypes = [ctypes.c_int]
    lib.pa_plan.restype = ctypes.c_int
    lib.pa_plan.argtypes = [ctypes.POINTER(BatchDesc), ctypes.POINTER(vp), ctypes.POINTER(sz)]
    lib.pa_plan_fixed.restype = ctypes.c_int
    lib.pa_plan_fixed.argtypes = [ctypes.POINTER(BatchDesc), ctypes.POINTER(FixedShape), ctypes.POINTER(vp),
                                  ctypes.POINTER(sz)]
    lib.pa_upload_metadata.restype = ctypes.c_int
    lib.pa_upload_metadata.argtypes = [vp, vp, sz, vp]
    lib.pa_plan_metadata_bytes.restype = sz
    lib.pa_plan_metadata_bytes.argtypes = [vp]
    lib.pa_plan_copy_metadata.restype = ctypes.c_int
    lib.pa_plan_copy_metadata.argtypes = [vp, vp, sz]
    lib.pa_upload_metadata_from.restype = ctypes.c_int
    lib.pa_upload_metadata_from.argtypes = [vp, sz, vp, sz, vp]
    lib.pa_graph_create.restype = ctypes.c_int
    lib.pa_graph_create.argtypes = [vp, vp, vp, ctypes.POINTER(vp)]
    lib.pa_graph_step.restype = ctypes.c_int
    lib.pa_graph_step.argtypes = [vp, vp, vp]
    lib.pa_graph_turn.restype = i32
    lib.pa_graph_turn.argtypes = [vp]
    lib.pa_graph_wait.restype = ctypes.c_int
    lib.pa_graph_wait.argtypes = [vp, i32]
    lib.pa_graph_workspace.restype = vp
    lib.pa_graph_workspace.argtypes = [vp]
    lib.pa_graph_slot_mapping.restype = vp
    lib.pa_graph_slot_mapping.argtypes = [vp]
    lib.pa_graph_destroy.restype = None
    lib.pa_graph_destroy.argtypes = [vp]
    lib.pa_attention_launch.restype = ctypes.c_int
    lib.pa_attention_launch.argtypes = [vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.pa_attention_with_kv_update.restype = ctypes.c_int
    lib.pa_attention_with_kv_update.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.pa_attention_with_kv_update_launch.restype = ctypes.c_int
    lib.pa_attention_with_kv_update_launch.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.pa_attention_with_kv_update_launch_staged.restype = ctypes.c_int
    lib.pa_attention_with_kv_update_launch_staged.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp, vp]
    lib.pa_zero_blocks.restype = ctypes.c_int
    lib.pa_zero_blocks.argtypes = [vp, i32, i32, i32, i32, i32, vp, vp, vp, vp]
    lib.pa_plan_destroy.restype = None
    lib.pa_plan_destroy.argtypes = [vp]
    lib.pa_plan_get_info.restype = ctypes.c_int
    lib.pa_plan_get_info.argtypes = [vp, ctypes.POINTER(PlanInfo)]
    lib.pa_slot_mapping.restype = ctypes.c_int
    lib.pa_slot_mapping.argtypes = [vp, vp, vp, i32, i32, i32, i32, vp, vp]
    lib.pa_write_kv.restype = ctypes.c_int
    lib.pa_write_kv.argtypes = [vp, vp, vp, i32, i32, i32, vp, vp, i64, vp, vp]
    lib.pa_write_kv_fp8.restype = ctypes.c_int
    lib.pa_write_kv_fp8.argtypes = [vp, vp, vp, i32, i32, i32, vp, vp, i64, ctypes.c_float, ctypes.c_float, vp, vp]
    lib.pa_attention.restype = ctypes.c_int
    lib.pa_attention.argtypes = [vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.pa_attention_no_alloc.restype = ctypes.c_int
    lib.pa_attention_no_alloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp]
    lib.pa_check_device_errors.restype = ctypes.c_int
    lib.pa_check_device_errors.argtypes = [vp, i32p, vp]
    lib.pa_plan_enable_timing.restype = ctypes.c_int
    lib.pa_plan_enable_timing.argtypes = [vp, i32]
    lib.pa_plan_kernel_times.restype = ctypes.c_int
    lib.pa_plan_kernel_times.argtypes = [vp, ctypes.POINTER(ctypes.c_double), i32p]
    lib.pa_rope_create.restype = ctypes.c_int
    lib.pa_rope_create.argtypes = [ctypes.POINTER(RopeDesc), ctypes.POINTER(vp)]
    lib.pa_rope_destroy.restype = None
    lib.pa_rope_destroy.argtypes = [vp]
    lib.pa_rope_frequencies.restype = ctypes.c_int
    lib.pa_rope_frequencies.argtypes = [vp, vp, vp]
    lib.pa_rotary.restype = ctypes.c_int
    lib.pa_rotary.argtypes = [vp, vp, i64, vp, i32, i32, i32, vp, i64, vp]
    lib.pa_append_kv.restype = ctypes.c_int
    lib.pa_append_kv.argtypes = [vp, ctypes.POINTER(AppendArgs), vp]
    lib.pa_attention_scaled.restype = ctypes.c_int
    lib.pa_attention_scaled.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.pa_attention_scaled_launch.restype = ctypes.c_int
    lib.pa_attention_scaled_launch.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.pa_plan_window.restype = ctypes.c_int
    lib.pa_plan_window.argtypes = [ctypes.POINTER(BatchDesc), ctypes.POINTER(WindowDesc), ctypes.POINTER(FixedShape),
                                   ctypes.POINTER(vp), ctypes.POINTER(sz)]
    lib.pa_rope_create_axes.restype = ctypes.c_int
    lib.pa_rope_create_axes.argtypes = [ctypes.POINTER(RopeDesc), ctypes.POINTER(RopeAxesDesc), ctypes.POINTER(vp)]
    lib.pa_rotary_axes.restype = ctypes.c_int
    lib.pa_rotary_axes.argtypes = [vp, vp, i64, vp, i64, i32, i32, i32, vp, i64, vp]
    lib.pa_append_kv_axes.restype = ctypes.c_int
    lib.pa_append_kv_axes.argtypes = [vp, ctypes.POINTER(AppendArgs), vp, i64, vp]
    if path is None:
        _LIB = lib
    return lib


def status_string(status: int) -> str:
    try:
        return load().pa_status_string(int(status)).decode()
    except RuntimeError:
        return f"status {status}"


def _check(status: int, what: str):
    if status != PA_OK:
        raise PaError(status, what)


def _ptr(t) -> int | None:
    """Raw device/host address of a tensor or an address (or None)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return int(t.data_ptr())


# What the calls that take tensors ask of torch, which the first of them imports:
# plans, their metadata and rotations need none.
_cuda = _raw_stream = _raw_device = _BF16 = _I32 = _F32 = None
_PLAIN_CACHES, _SCALED_CACHES = {}, {}


def _use_torch():
    global _cuda, _raw_stream, _raw_device, _BF16, _I32, _F32
    import torch
    _PLAIN_CACHES.update({torch.bfloat16: PA_KV_BF16, torch.uint8: PA_KV_FP8_E4M3})
    _SCALED_CACHES.update({torch.uint8: PA_KV_FP8_E4M3_BLOCK, torch.int8: PA_KV_INT8_BLOCK})
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    _raw_device = getattr(torch._C, "_cuda_getDevice", None)
    _BF16, _I32, _F32 = torch.bfloat16, torch.int32, torch.float32
    _cuda = torch.cuda


def _stream(stream) -> int | None:
    if stream is None:
        if _cuda is None:
            _use_torch()
        # the current stream's handle without a Stream object (0.2 us against
        # 2.9: as long as the C call itself)
        if _raw_stream is not None and _raw_device is not None and _cuda.is_initialized():
            return _raw_stream(_raw_device())
        return int(_cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


@dataclass
class Plan:
    handle: int
    workspace_bytes: int
    _keep: tuple  # host arrays referenced while pa_plan runs
    # what the tensors of its calls have to be: (kv_cache_dtype, elements of q and
    # out, num_blocks, kv heads, head_dim, elements of the block table, its width)
    _step: tuple | None = None
    window: tuple | None = None   # (window, sink_tokens) of pa_plan_window
    heads_q: int = 0              # with a window

    def info(self) -> dict:
        pi = PlanInfo()
        _check(load().pa_plan_get_info(self.handle, ctypes.byref(pi)), "pa_plan_get_info")
        return pi.as_dict()

    def enable_timing(self, on: bool = True):
        _check(load().pa_plan_enable_timing(self.handle, 1 if on else 0), "pa_plan_enable_timing")

    def kernel_times(self):
        ms = (ctypes.c_double * 4)()
        n = (ctypes.c_int32 * 4)()
        _check(load().pa_plan_kernel_times(self.handle, ms, n), "pa_plan_kernel_times")
        return list(ms), list(n)

    def destroy(self):
        if self.handle:
            load().pa_plan_destroy(self.handle)
            self.handle = 0

    def __del__(self):
        try:
            self.destroy()
        except Exception:  # noqa: BLE001 -- interpreter shutdown
            pass


def make_desc(*, num_heads_q, num_heads_kv, head_dim, num_blocks, query_start_loc, seq_lens,
              num_computed_tokens, block_table_host=None, max_blocks_per_req=None,
              num_common_prefix_blocks=0, softmax_scale, num_sms=0, block_size=16, kv_cache_dtype=0,
              k_scale=1.0, v_scale=1.0):
    qsl = np.ascontiguousarray(query_start_loc, dtype=np.int32)
    sl = np.ascontiguousarray(seq_lens, dtype=np.int32)
    nc = np.ascontiguousarray(num_computed_tokens, dtype=np.int32)
    bt = None if block_table_host is None else np.ascontiguousarray(block_table_host, dtype=np.int32)
    if max_blocks_per_req is None:
        max_blocks_per_req = bt.shape[1] if bt is not None else 1
    d = BatchDesc(len(sl), num_heads_q, num_heads_kv, head_dim, block_size, num_blocks, int(max_blocks_per_req),
                  qsl.ctypes.data, sl.ctypes.data, nc.ctypes.data, bt.ctypes.data if bt is not None else None,
                  int(num_common_prefix_blocks), float(softmax_scale), int(num_sms), int(kv_cache_dtype),
                  float(k_scale), float(v_scale))
    return d, (qsl, sl, nc, bt)


def _step_of(d: BatchDesc, rows: int) -> tuple:
    return (d.kv_cache_dtype, rows * d.num_heads_q * d.head_dim, d.num_blocks, d.num_heads_kv, d.head_dim,
            d.num_reqs * d.max_blocks_per_req, d.max_blocks_per_req)


def pa_plan(**kw) -> Plan:
    """Validate the step's metadata and build its plan (see pa.h)."""
    d, keep = make_desc(**kw)
    handle = ctypes.c_void_p()
    ws = ctypes.c_size_t()
    _check(load().pa_plan(ctypes.byref(d), ctypes.byref(handle), ctypes.byref(ws)), "pa_plan")
    return Plan(handle.value, ws.value, keep, _step_of(d, int(keep[0][-1]) if len(keep[0]) else 0))


def _fixed_shape(max_tokens, max_reqs, max_extend_tiles=0, max_dequant_blocks=0, max_partial_slots=0,
                 decode_prefix_tokens=0):
    fs = FixedShape()
    fs.max_tokens, fs.max_reqs = int(max_tokens), int(max_reqs)
    fs.max_extend_tiles, fs.max_dequant_blocks = int(max_extend_tiles), int(max_dequant_blocks)
    fs.max_partial_slots = int(max_partial_slots)
    fs.decode_prefix_tokens = int(decode_prefix_tokens)
    return fs


def pa_plan_fixed(*, max_tokens, max_reqs, max_extend_tiles=0, max_dequant_blocks=0, max_partial_slots=0,
                  decode_prefix_tokens=0, **kw) -> Plan:
    """A fixed-shape plan (graph-capturable launches, see pa.h)."""
    d, keep = make_desc(**kw)
    fs = _fixed_shape(max_tokens, max_reqs, max_extend_tiles, max_dequant_blocks, max_partial_slots,
                      decode_prefix_tokens)
    handle = ctypes.c_void_p()
    ws = ctypes.c_size_t()
    _check(load().pa_plan_fixed(ctypes.byref(d), ctypes.byref(fs), ctypes.byref(handle), ctypes.byref(ws)),
           "pa_plan_fixed")
    return Plan(handle.value, ws.value, keep, _step_of(d, fs.max_tokens))


def pa_plan_fixed_status(*, max_tokens, max_reqs, max_extend_tiles=0, max_dequant_blocks=0, max_partial_slots=0,
                         decode_prefix_tokens=0, **kw) -> int:
    """Status code pa_plan_fixed returns (plan discarded)."""
    d, keep = make_desc(**kw)
    fs = _fixed_shape(max_tokens, max_reqs, max_extend_tiles, max_dequant_blocks, max_partial_slots,
                      decode_prefix_tokens)
    handle = ctypes.c_void_p()
    ws = ctypes.c_size_t()
    st = load().pa_plan_fixed(ctypes.byref(d), ctypes.byref(fs), ctypes.byref(handle), ctypes.byref(ws))
    if st == PA_OK:
        load().pa_plan_destroy(handle.value)
    return st


def _int32(n) -> int:
    """For a 32-bit field that holds no negative number: one that it does not hold is
    refused like those (ctypes would wrap it)."""
    n = int(n)
    return n if -2**31 <= n < 2**31 else -1


def _plan_window(window, sink_tokens, shape, kw):
    window, sink_tokens = _int32(window), _int32(sink_tokens)
    d, keep = make_desc(**kw)
    fs = _fixed_shape(**shape) if shape else None
    handle = ctypes.c_void_p()
    ws = ctypes.c_size_t()
    st = load().pa_plan_window(ctypes.byref(d), ctypes.byref(WindowDesc(window, sink_tokens)),
                               ctypes.byref(fs) if fs is not None else None, ctypes.byref(handle), ctypes.byref(ws))
    rows = fs.max_tokens if fs is not None else int(keep[0][-1]) if len(keep[0]) else 0
    return st, handle.value, lambda: Plan(handle.value, ws.value, keep, _step_of(d, rows), (window, sink_tokens),
                                          d.num_heads_q)


def pa_plan_window(*, window, sink_tokens=0, shape: dict | None = None, **kw) -> Plan:
    """A plan whose queries see the last ``window`` keys and the first
    ``sink_tokens`` (see pa.h); ``shape``: the arguments of pa_plan_fixed for a
    fixed-shape plan."""
    st, _, plan = _plan_window(window, sink_tokens, shape, kw)
    _check(st, "pa_plan_window")
    return plan()


def pa_plan_window_status(*, window, sink_tokens=0, shape: dict | None = None, **kw) -> int:
    """Status code pa_plan_window returns (plan discarded)."""
    st, handle, _ = _plan_window(window, sink_tokens, shape, kw)
    if st == PA_OK:
        load().pa_plan_destroy(handle)
    return st


def pa_plan_status(**kw) -> int:
    """Status code pa_plan returns for this descriptor (plan discarded)."""
    d, keep = make_desc(**kw)
    handle = ctypes.c_void_p()
    ws = ctypes.c_size_t()
    st = load().pa_plan(ctypes.byref(d), ctypes.byref(handle), ctypes.byref(ws))
    if st == PA_OK:
        load().pa_plan_destroy(handle.value)
    return st


def pa_slot_mapping(query_start_loc, num_computed, block_table, num_tokens: int, slot_mapping,
                    block_size: int = 16, stream=None):
    _check(load().pa_slot_mapping(_ptr(query_start_loc), _ptr(num_computed), _ptr(block_table),
                                  int(num_computed.numel()), int(num_tokens), int(block_table.shape[1]),
                                  int(block_size), _ptr(slot_mapping), _stream(stream)), "pa_slot_mapping")


def pa_write_kv(key, value, slot_mapping, key_cache, value_cache, device_error_word=None, stream=None):
    T, hkv, d = key.shape
    num_slots = key_cache.shape[0] * key_cache.shape[1]
    _check(load().pa_write_kv(_ptr(key), _ptr(value), _ptr(slot_mapping), T, hkv, d, _ptr(key_cache),
                              _ptr(value_cache), num_slots, _ptr(device_error_word), _stream(stream)),
           "pa_write_kv")


def pa_write_kv_fp8(key, value, slot_mapping, key_cache, value_cache, k_scale: float, v_scale: float,
                    device_error_word=None, stream=None):
    """Quantising cache write into E4M3 caches (uint8 tensors)."""
    T, hkv, d = key.shape
    num_slots = key_cache.shape[0] * key_cache.shape[1]
    _check(load().pa_write_kv_fp8(_ptr(key), _ptr(value), _ptr(slot_mapping), T, hkv, d, _ptr(key_cache),
                                  _ptr(value_cache), num_slots, float(k_scale), float(v_scale),
                                  _ptr(device_error_word), _stream(stream)), "pa_write_kv_fp8")


def _check_window(plan, q, key_cache, value_cache, block_table, out, *more):
    """Windowed plans: the kernels go by the plan, so tensors of another step, type or
    device would be read as what they are not, or past their ends."""
    if _cuda is None:
        _use_torch()
    # (element counts: a shape object costs as much as three other questions, and
    # the smallest calls are bound by this thread)
    kind, rows, nb, hkv, dim, entries, width = plan._step
    dtype = key_cache.dtype
    blocks, slots, heads, d = key_cache.shape
    if _PLAIN_CACHES.get(dtype) != kind or value_cache.dtype is not dtype or slots != 16 or heads != hkv or d != dim or \
            blocks < nb or value_cache.numel() != key_cache.numel() or not key_cache.is_contiguous() or \
            not value_cache.is_contiguous():
        raise ValueError(f"caches: the plan's type, contiguous [{nb}, 16, {hkv}, {dim}] wanted")
    if q.dtype is not _BF16 or out.dtype is not _BF16 or q.numel() < rows or out.numel() < rows or \
            not q.is_contiguous() or not out.is_contiguous():
        raise ValueError(f"q, out: contiguous bf16, all of the plan's rows wanted ({rows} elements)")
    if block_table.dtype is not _I32 or not block_table.is_contiguous() or block_table.numel() < entries or \
            block_table.shape[-1] != width:
        raise ValueError(f"block_table: contiguous int32, the plan's requests and its {width} blocks each wanted")
    _here("q, caches, block table, out, workspace", q, key_cache, value_cache, block_table, out, *more)


def _check_new_rows(plan, key, value, slot_mapping):
    """The new rows of a fused call with a windowed plan."""
    import torch
    _, rows, _, hkv, dim, _, _ = plan._step
    tokens = rows // (plan.heads_q * dim)
    need = tokens * hkv * dim
    for t in (key, value):
        if t.dtype is not _BF16 or not t.is_contiguous() or t.numel() < need:
            raise ValueError(f"key, value: contiguous bf16, all of the plan's rows wanted ({need} elements)")
    if slot_mapping is not None and (slot_mapping.dtype is not torch.int64 or slot_mapping.numel() < tokens or
                                     not slot_mapping.is_contiguous()):
        raise ValueError("slot_mapping: contiguous int64, one per row of the plan wanted")
    if slot_mapping is not None:
        _here("slot_mapping", slot_mapping)


def pa_attention(plan: Plan, q, key_cache, value_cache, block_table, out, workspace, stream=None):
    if plan.window is not None:
        _check_window(plan, q, key_cache, value_cache, block_table, out, workspace)
    nbytes = workspace.numel() * workspace.element_size()
    _check(load().pa_attention(plan.handle, _ptr(q), _ptr(key_cache), _ptr(value_cache), _ptr(block_table),
                               _ptr(out), _ptr(workspace), nbytes, _stream(stream)), "pa_attention")


def pa_upload_metadata(plan: Plan, workspace, stream=None):
    nbytes = workspace.numel() * workspace.element_size()
    _check(load().pa_upload_metadata(plan.handle, _ptr(workspace), nbytes, _stream(stream)), "pa_upload_metadata")


def pa_plan_metadata_bytes(plan: Plan) -> int:
    return int(load().pa_plan_metadata_bytes(plan.handle))


def pa_plan_copy_metadata_status(plan: Plan, host_dst, nbytes: int) -> int:
    """Raw status of pa_plan_copy_metadata into host memory at address host_dst."""
    return load().pa_plan_copy_metadata(plan.handle, host_dst, nbytes)


def pa_plan_copy_metadata(plan: Plan, host_dst):
    """Copy the plan's metadata image into a host tensor (uint8, at least
    pa_plan_metadata_bytes long)."""
    nbytes = host_dst.numel() * host_dst.element_size()
    _check(pa_plan_copy_metadata_status(plan, _ptr(host_dst), nbytes), "pa_plan_copy_metadata")


def pa_upload_metadata_from(host_src, nbytes: int, workspace, stream=None):
    """Enqueue the upload of a metadata image from page-locked host memory
    (capturable; see pa.h)."""
    wbytes = workspace.numel() * workspace.element_size()
    _check(load().pa_upload_metadata_from(_ptr(host_src), nbytes, _ptr(workspace), wbytes, _stream(stream)),
           "pa_upload_metadata_from")


def pa_attention_launch(plan: Plan, q, key_cache, value_cache, block_table, out, workspace, stream=None):
    """The attention kernels alone (capturable in a CUDA graph; see pa.h)."""
    if plan.window is not None:
        _check_window(plan, q, key_cache, value_cache, block_table, out, workspace)
        st = load().pa_attention_launch(plan.handle, q.data_ptr(), key_cache.data_ptr(), value_cache.data_ptr(),
                                        block_table.data_ptr(), out.data_ptr(), workspace.data_ptr(), workspace.nbytes,
                                        _stream(stream))
        if st:
            _check(st, "pa_attention_launch")
        return
    nbytes = workspace.numel() * workspace.element_size()
    _check(load().pa_attention_launch(plan.handle, _ptr(q), _ptr(key_cache), _ptr(value_cache), _ptr(block_table),
                                      _ptr(out), _ptr(workspace), nbytes, _stream(stream)), "pa_attention_launch")


def pa_attention_with_kv_update(plan: Plan, q, key, value, key_cache, value_cache, block_table, out, workspace,
                                slot_mapping=None, stream=None):
    """Cache write + attention in one call (see pa.h)."""
    if plan.window is not None:
        _check_window(plan, q, key_cache, value_cache, block_table, out, workspace, key, value)
        _check_new_rows(plan, key, value, slot_mapping)
    nbytes = workspace.numel() * workspace.element_size()
    _check(load().pa_attention_with_kv_update(plan.handle, _ptr(q), _ptr(key), _ptr(value), _ptr(key_cache),
                                              _ptr(value_cache), _ptr(block_table), _ptr(slot_mapping), _ptr(out),
                                              _ptr(workspace), nbytes, _stream(stream)),
           "pa_attention_with_kv_update")


def pa_attention_with_kv_update_launch(plan: Plan, q, key, value, key_cache, value_cache, block_table, out,
                                       workspace, slot_mapping=None, stream=None):
    if plan.window is not None:
        _check_window(plan, q, key_cache, value_cache, block_table, out, workspace, key, value)
        _check_new_rows(plan, key, value, slot_mapping)
    nbytes = workspace.numel() * workspace.element_size()
    _check(load().pa_attention_with_kv_update_launch(plan.handle, _ptr(q), _ptr(key), _ptr(value), _ptr(key_cache),
                                                     _ptr(value_cache), _ptr(block_table), _ptr(slot_mapping),
                                                     _ptr(out), _ptr(workspace), nbytes, _stream(stream)),
           "pa_attention_with_kv_update_launch")


def pa_attention_with_kv_update_launch_staged(plan: Plan, q, key, value, key_cache, value_cache, block_table, out,
                                              workspace, late_rows, slot_mapping=None, stream=None,
                                              late_out_ready=None):
    """As pa_attention_with_kv_update_launch; rows from the plan's decode
    prefix on may still be written until late_rows (a torch.cuda.Event,
    already recorded) fires.  late_out_ready (a torch.cuda.Event) is recorded
    once out's rows from the prefix on are final."""
    if plan.window is not None:
        _check_window(plan, q, key_cache, value_cache, block_table, out, workspace, key, value)
        _check_new_rows(plan, key, value, slot_mapping)
    nbytes = workspace.numel() * workspace.element_size()
    if late_out_ready is not None and not late_out_ready.cuda_event:
        late_out_ready.record()   # torch creates the CUDA event at its first record
    _check(load().pa_attention_with_kv_update_launch_staged(
        plan.handle, _ptr(q), _ptr(key), _ptr(value), _ptr(key_cache), _ptr(value_cache), _ptr(block_table),
        _ptr(slot_mapping), _ptr(out), _ptr(workspace), nbytes, _stream(stream),
        ctypes.c_void_p(late_rows.cuda_event if late_rows is not None else 0),
        ctypes.c_void_p(late_out_ready.cuda_event if late_out_ready is not None else 0)),
        "pa_attention_with_kv_update_launch_staged")


def pa_zero_blocks(block_ids, key_cache, value_cache, device_error_word=None, stream=None):
    """Zero the K and V entries of the listed blocks (ids < 0 skipped)."""
    nb, bs, hkv, d = key_cache.shape
    kv = PA_KV_FP8_E4M3 if key_cache.element_size() == 1 else PA_KV_BF16
    _check(load().pa_zero_blocks(_ptr(block_ids), int(block_ids.numel()), nb, hkv, d, kv, _ptr(key_cache),
                                 _ptr(value_cache), _ptr(device_error_word), _stream(stream)), "pa_zero_blocks")


def pa_attention_no_alloc(plan: Plan, q, key_cache, value_cache, block_table, out, device_error_word=None,
                          stream=None):
    """pa_attention with the library's fixed scratch array instead of a workspace
    (for callers that cannot allocate device memory; see pa.h)."""
    if plan.window is not None:
        more = () if device_error_word is None or isinstance(device_error_word, int) else (device_error_word,)
        _check_window(plan, q, key_cache, value_cache, block_table, out, *more)
    _check(load().pa_attention_no_alloc(plan.handle, _ptr(q), _ptr(key_cache), _ptr(value_cache),
                                        _ptr(block_table), _ptr(out), _ptr(device_error_word), _stream(stream)),
           "pa_attention_no_alloc")


@dataclass
class Rope:
    """pa_rope_t: a rotation by position (see pa.h); immutable, used by any
    number of calls, streams and captured graphs."""
    handle: int
    rotary_dim: int
    num_axes: int = 1

    def frequencies(self):
        """(angles per position [rotary_dim / 2] as float64, factor on cos and sin)"""
        f = np.empty(self.rotary_dim // 2, dtype=np.float64)
        m = ctypes.c_double()
        _check(load().pa_rope_frequencies(self.handle, f.ctypes.data, ctypes.addressof(m)), "pa_rope_frequencies")
        return f, m.value

    def destroy(self):
        if self.handle:
            load().pa_rope_destroy(self.handle)
            self.handle = 0

    def __del__(self):
        try:
            self.destroy()
        except Exception:  # noqa: BLE001 -- interpreter shutdown
            pass


def _rope_desc(rotary_dim, layout, base, scaling, factor, original_max_position, low, high, attention_factor):
    return RopeDesc(int(rotary_dim), int(layout), int(scaling), int(original_max_position), float(base), float(factor),
                    float(low), float(high), float(attention_factor))


def pa_rope_create(*, rotary_dim, layout=PA_ROPE_HALF, base=10000.0, scaling=PA_ROPE_SCALE_NONE, factor=1.0,
                   original_max_position=0, low=1.0, high=4.0, attention_factor=0.0) -> Rope:
    """Build a rotation (host only, see pa.h)."""
    d = _rope_desc(rotary_dim, layout, base, scaling, factor, original_max_position, low, high, attention_factor)
    h = ctypes.c_void_p()
    _check(load().pa_rope_create(ctypes.byref(d), ctypes.byref(h)), "pa_rope_create")
    return Rope(h.value, int(rotary_dim))


def pa_rope_status(*, rotary_dim, layout=PA_ROPE_HALF, base=10000.0, scaling=PA_ROPE_SCALE_NONE, factor=1.0,
                   original_max_position=0, low=1.0, high=4.0, attention_factor=0.0) -> int:
    """Status code pa_rope_create returns (rotation discarded)."""
    d = _rope_desc(rotary_dim, layout, base, scaling, factor, original_max_position, low, high, attention_factor)
    h = ctypes.c_void_p()
    st = load().pa_rope_create(ctypes.byref(d), ctypes.byref(h))
    if st == PA_OK:
        load().pa_rope_destroy(h.value)
    return st


def _axes_desc(rotary_dim, num_axes, axis_of_pair, frequencies):
    given = np.asarray(axis_of_pair)
    with np.errstate(invalid="ignore"):   # (a number that 32 bits do not hold comes out as another)
        axis = np.ascontiguousarray(given.astype(np.int32))
    if axis.ndim != 1 or 2 * axis.size != rotary_dim or (axis != given).any():
        raise ValueError("axis_of_pair: an axis for each of the rotary_dim / 2 pairs wanted")
    return RopeAxesDesc(_int32(num_axes), _int32(frequencies), axis.ctypes.data), axis


def pa_rope_create_axes(*, num_axes, axis_of_pair, rotary_dim, frequencies=PA_ROPE_AXES_SHARED, layout=PA_ROPE_HALF,
                        base=10000.0, scaling=PA_ROPE_SCALE_NONE, factor=1.0, original_max_position=0, low=1.0, high=4.0,
                        attention_factor=0.0) -> Rope:
    """Build a rotation with positions on several axes (host only, see pa.h)."""
    d = _rope_desc(rotary_dim, layout, base, scaling, factor, original_max_position, low, high, attention_factor)
    axes, _keep = _axes_desc(rotary_dim, num_axes, axis_of_pair, frequencies)
    h = ctypes.c_void_p()
    _check(load().pa_rope_create_axes(ctypes.byref(d), ctypes.byref(axes), ctypes.byref(h)), "pa_rope_create_axes")
    return Rope(h.value, int(rotary_dim), int(num_axes))


def _axis_stride(rope: Rope, positions, num_tokens: int) -> int:
    """Elements between the axes of positions (int32 [axes, tokens], tokens dense)."""
    n = rope.num_axes
    if positions.dtype is not _I32 or positions.shape != (n, num_tokens):
        raise ValueError(f"positions: int32 [{n}, {num_tokens}] wanted")
    apart, dense = positions.stride()
    if num_tokens > 1 and dense != 1:
        raise ValueError("positions: dense rows wanted")
    return num_tokens if n == 1 else apart


def _here(what: str, *tensors):
    """Refuse tensors that kernels on the current device cannot read (one left
    on the host among them)."""
    device = tensors[0].get_device()   # (-1: the host)
    if device >= 0 and device == (_raw_device or _cuda.current_device)():
        for t in tensors:
            if t.get_device() != device:
                break
        else:
            return
    raise ValueError(f"{what}: tensors of the current CUDA device wanted")


def _rows(t, d: int, name: str) -> int:
    """Token stride of bf16 rows [tokens, heads, d] with dense heads (views of
    a packed projection output are)."""
    s = t.stride()
    if t.dtype is not _BF16 or len(s) != 3 or s[2] != 1 or s[1] != d:
        raise ValueError(f"{name}: bf16 rows [tokens, heads, {d}] with dense heads wanted")
    return s[0]


def pa_rotary(rope: Rope, x, positions, out, stream=None):
    """out = x (bf16 [T, H, D], token stride free) rotated by positions (int32
    [T]); out may be x."""
    if _cuda is None:
        _use_torch()
    shape = T, H, D = x.shape
    xs, os_ = _rows(x, D, "x"), _rows(out, D, "out")
    if out.shape != shape or positions.dtype is not _I32 or positions.numel() != T or not positions.is_contiguous():
        raise ValueError("out: x's shape wanted; positions: contiguous int32 [tokens]")
    _here("x, positions, out", x, positions, out)
    if T <= 1:   # a single row's stride is anything
        xs = os_ = H * D
    st = load().pa_rotary(rope.handle, x.data_ptr(), xs, positions.data_ptr(), T, H, D, out.data_ptr(), os_, _stream(stream))
    if st:
        _check(st, "pa_rotary")


def pa_rotary_axes(rope: Rope, x, positions, out, stream=None):
    """out = x (bf16 [T, H, D], token stride free) rotated by positions on the
    rotation's axes (int32 [axes, T]; a row expanded to them counts for all); out
    may be x."""
    if _cuda is None:
        _use_torch()
    shape = T, H, D = x.shape
    xs, os_ = _rows(x, D, "x"), _rows(out, D, "out")
    if out.shape != shape:
        raise ValueError("out: x's shape wanted")
    apart = _axis_stride(rope, positions, T)
    _here("x, positions, out", x, positions, out)
    if T <= 1:   # a single row's stride is anything
        xs = os_ = H * D
    st = load().pa_rotary_axes(rope.handle, x.data_ptr(), xs, positions.data_ptr(), apart, T, H, D, out.data_ptr(), os_,
                               _stream(stream))
    if st:
        _check(st, "pa_rotary_axes")


def _append_args(rope, key, value, query_start_loc, num_computed, block_table, key_cache, value_cache, key_scales,
                 value_scales, k_scale, v_scale, q, q_out, device_error_word):
    if rope is not None and not rope.handle:   # (without a rotation keys would be stored as they are)
        raise ValueError("rope: destroyed")
    if _cuda is None:
        _use_torch()
    shape = T, hkv, d = key.shape
    ks, vs = _rows(key, d, "key"), _rows(value, d, "value")
    pool, dtype = key_cache.shape, key_cache.dtype
    nb, bs = pool[0], pool[1]
    if value.shape != shape or pool != (nb, bs, hkv, d) or value_cache.shape != pool or value_cache.dtype is not dtype or \
            not key_cache.is_contiguous() or not value_cache.is_contiguous():
        raise ValueError(f"value: key's shape wanted; caches: contiguous [num_blocks, block_size, {hkv}, {d}] of one type")
    ksc = vsc = 0
    if key_scales is not None and value_scales is not None:
        kind = _SCALED_CACHES.get(dtype)
        if key_scales.dtype is not _F32 or value_scales.dtype is not _F32 or key_scales.shape != (nb, hkv) or \
                value_scales.shape != (nb, hkv) or not key_scales.is_contiguous() or not value_scales.is_contiguous():
            raise ValueError(f"scales: contiguous float [{nb}, {hkv}] wanted")
        ksc, vsc = key_scales.data_ptr(), value_scales.data_ptr()
    else:
        kind = _PLAIN_CACHES.get(dtype) if key_scales is value_scales else None
    if kind is None:
        raise ValueError(f"caches of {dtype} with these scales are none of PA_KV_*")
    R, mb = block_table.shape
    if num_computed.dtype is not _I32 or query_start_loc.dtype is not _I32 or block_table.dtype is not _I32 or \
            num_computed.numel() != R or query_start_loc.numel() != R + 1 or not block_table.is_contiguous() or \
            not num_computed.is_contiguous() or not query_start_loc.is_contiguous():
        raise ValueError("query_start_loc [R + 1], num_computed [R], block_table [R, blocks]: contiguous int32 wanted")
    hq = qp = qs = op = os_ = 0
    if q is not None and q_out is not None:
        hq, qp, op = q.shape[1], q.data_ptr(), q_out.data_ptr()
        qs, os_ = _rows(q, d, "q"), _rows(q_out, d, "q_out")
        if q.shape != (T, hq, d) or q_out.shape != (T, hq, d):
            raise ValueError(f"q, q_out: rows [{T}, heads, {d}] wanted")
    elif q is not q_out:
        raise ValueError("q and q_out come together")
    word = _ptr(device_error_word)
    if word is not None and word is not device_error_word and \
            (device_error_word.dtype is not _I32 or device_error_word.numel() < 1):
        raise ValueError("device_error_word: an int32 wanted")
    _here("rows, starts, lengths, block table, caches", key, value, query_start_loc, num_computed, block_table, key_cache,
          value_cache)
    if ksc:
        _here("scales", key_scales, value_scales)
    if qp:
        _here("q, q_out", q, q_out)
    if word is not None and word is not device_error_word:
        _here("device_error_word", device_error_word)
    if T <= 1:   # a single row's stride is anything
        ks = vs = hkv * d
        qs = os_ = hq * d
    return AppendArgs(R, T, hq, hkv, d, bs, nb, mb, kind, k_scale, v_scale, query_start_loc.data_ptr(), num_computed.data_ptr(),
                      block_table.data_ptr(), key.data_ptr(), value.data_ptr(), ks, vs, qp, op, qs, os_, key_cache.data_ptr(),
                      value_cache.data_ptr(), ksc, vsc, word)


def pa_append_kv(rope: Rope | None, key, value, query_start_loc, num_computed, block_table, key_cache, value_cache, *,
                 key_scales=None, value_scales=None, k_scale: float = 1.0, v_scale: float = 1.0, q=None, q_out=None,
                 device_error_word=None, stream=None):
    """The cache write with the rotation of key (and q into q_out) on the way
    (see pa.h).  The cache's type follows from the tensors: bf16; uint8 E4M3
    codes with k_scale / v_scale; uint8 or int8 codes with key_scales and
    value_scales (float [num_blocks, Hkv])."""
    a = _append_args(rope, key, value, query_start_loc, num_computed, block_table, key_cache, value_cache, key_scales,
                     value_scales, k_scale, v_scale, q, q_out, device_error_word)
    st = load().pa_append_kv(rope.handle if rope is not None else None, a, _stream(stream))
    if st:
        _check(st, "pa_append_kv")


def pa_append_kv_axes(rope: Rope, key, value, positions, query_start_loc, num_computed, block_table, key_cache,
                      value_cache, *, key_scales=None, value_scales=None, k_scale: float = 1.0, v_scale: float = 1.0,
                      q=None, q_out=None, device_error_word=None, stream=None):
    """pa_append_kv with rows rotated by positions of their own (int32 [axes, T],
    see pa.h)."""
    a = _append_args(rope, key, value, query_start_loc, num_computed, block_table, key_cache, value_cache, key_scales,
                     value_scales, k_scale, v_scale, q, q_out, device_error_word)
    apart = _axis_stride(rope, positions, key.shape[0])
    _here("rows, positions", key, positions)
    st = load().pa_append_kv_axes(rope.handle, a, positions.data_ptr(), apart, _stream(stream))
    if st:
        _check(st, "pa_append_kv_axes")


def _attention_args(plan, q, key_cache, value_cache, key_scales, value_scales, block_table, out, workspace):
    if _cuda is None:
        _use_torch()
    # (element counts: a shape object costs as much as three other questions, and
    # the smallest calls are bound by this thread)
    blocks, slots, heads, d = key_cache.shape
    n = blocks * heads
    if key_scales.dtype is not _F32 or value_scales.dtype is not _F32 or key_scales.numel() != n or \
            value_scales.numel() != n or not key_scales.is_contiguous() or not value_scales.is_contiguous():
        raise ValueError(f"scales: contiguous float [{blocks}, {heads}] wanted")
    if q.dtype is not _BF16 or out.dtype is not _BF16 or not q.is_contiguous() or not out.is_contiguous():
        raise ValueError("q, out: contiguous bf16 wanted")
    if block_table.dtype is not _I32 or not block_table.is_contiguous():
        raise ValueError("block_table: contiguous int32 wanted")
    codes = key_cache.dtype
    code_kind = _SCALED_CACHES.get(codes)
    if code_kind is None or value_cache.dtype is not codes or value_cache.numel() != n * slots * d or \
            not key_cache.is_contiguous() or not value_cache.is_contiguous():
        raise ValueError("caches: contiguous codes (uint8 or int8) of one shape wanted")
    if plan is not None and plan._step is not None:
        # the kernels go by the plan: tensors of another step, or codes of another
        # type, would be read as what they are not, or past their ends
        kind, rows, nb, hkv, dim, entries, width = plan._step
        if code_kind != kind:
            raise ValueError("caches: the type of codes that the plan was made for wanted")
        if heads != hkv or d != dim or blocks < nb or slots != 16:
            raise ValueError(f"caches: the plan's [{nb}, 16, {hkv}, {dim}] wanted")
        if q.numel() < rows or out.numel() < rows:
            raise ValueError(f"q, out: all of the plan's rows wanted ({rows} elements)")
        if block_table.numel() < entries or block_table.shape[-1] != width:
            raise ValueError(f"block_table: the plan's requests and its {width} blocks each wanted")
    _here("q, caches, scales, block table, out, workspace", q, key_cache, value_cache, key_scales, value_scales,
          block_table, out, workspace)


def pa_attention_scaled(plan: Plan, q, key_cache, value_cache, key_scales, value_scales, block_table, out, workspace,
                        stream=None):
    """Attention over block-scaled 8-bit caches (see pa.h)."""
    _attention_args(plan, q, key_cache, value_cache, key_scales, value_scales, block_table, out, workspace)
    st = load().pa_attention_scaled(plan.handle, q.data_ptr(), key_cache.data_ptr(), value_cache.data_ptr(),
                                    key_scales.data_ptr(), value_scales.data_ptr(), block_table.data_ptr(),
                                    out.data_ptr(), workspace.data_ptr(), workspace.nbytes, _stream(stream))
    if st:
        _check(st, "pa_attention_scaled")


def pa_attention_scaled_launch(plan: Plan, q, key_cache, value_cache, key_scales, value_scales, block_table, out,
                               workspace, stream=None):
    """Its kernels alone, after pa_upload_metadata (capturable in a CUDA graph)."""
    _attention_args(plan, q, key_cache, value_cache, key_scales, value_scales, block_table, out, workspace)
    st = load().pa_attention_scaled_launch(plan.handle, q.data_ptr(), key_cache.data_ptr(), value_cache.data_ptr(),
                                           key_scales.data_ptr(), value_scales.data_ptr(), block_table.data_ptr(),
                                           out.data_ptr(), workspace.data_ptr(), workspace.nbytes, _stream(stream))
    if st:
        _check(st, "pa_attention_scaled_launch")


NO_ALLOC_SCRATCH_BYTES = 16 << 20


def pa_check_device_errors(word, stream=None) -> int:
    """Read and clear a device error word; returns the PA_DEVERR_* bits seen."""
    bits = ctypes.c_int32(0)
    st = load().pa_check_device_errors(_ptr(word), ctypes.byref(bits), _stream(stream))
    if st not in (PA_OK, PA_ERR_DEVICE_CHECK):
        raise PaError(st, "pa_check_device_errors")
    return int(bits.value)


class NativeGraph:
    """pa_graph_t: the two captured step graphs of one fixed shape (see pa.h).

    ``host``: the step's metadata arrays the planner reads each step
    (query_start_loc [max_reqs+1], seq_lens [max_reqs], num_computed
    [max_reqs], block_table [max_reqs][max_blocks_per_req], int32 numpy
    arrays kept by the caller and rewritten in place), or a pair of such sets,
    one per graph (step n reads set ``turn``); ``num_reqs`` is set per step.
    ``buffers``: the device (and optional page-locked host I/O) buffers of
    pa_graph_buffers, as tensors or raw addresses.
    """

    def __init__(self, *, shape: dict, host: dict, buffers: dict, num_reqs: int, fused: bool, **model):
        sets = list(host) if isinstance(host, (list, tuple)) else [host, host]
        self._host = sets
        self._descs = []
        for hs in sets:
            for k in ("query_start_loc", "seq_lens", "num_computed", "block_table"):
                a = hs[k]
                if not (isinstance(a, np.ndarray) and a.dtype == np.int32 and a.flags.c_contiguous):
                    raise ValueError(f"host[{k!r}] must be a C-contiguous int32 numpy array")
            d, _ = make_desc(query_start_loc=hs["query_start_loc"], seq_lens=hs["seq_lens"],
                             num_computed_tokens=hs["num_computed"], block_table_host=hs["block_table"], **model)
            # the descriptor points into the caller's arrays, rewritten each step
            d.query_start_loc = hs["query_start_loc"].ctypes.data
            d.seq_lens = hs["seq_lens"].ctypes.data
            d.num_computed_tokens = hs["num_computed"].ctypes.data
            d.block_table_host = hs["block_table"].ctypes.data
            d.num_reqs = int(num_reqs)
            self._descs.append(d)
        self._shape = _fixed_shape(**shape)
        addr = lambda t: None if t is None else (t if isinstance(t, int) else int(t.data_ptr()))  # noqa: E731
        b = GraphBuffers()
        for k in ("q", "key", "value", "out", "query_start_loc", "num_computed", "block_table", "key_cache",
                  "value_cache", "device_in"):
            setattr(b, k, addr(buffers.get(k)))
        b.fused = 1 if fused else 0
        for k, n in (("host_in", "in_bytes"), ("host_out", "out_bytes")):
            pair = buffers.get(k)
            if pair is not None:
                getattr(b, k)[0] = addr(pair[0])
                getattr(b, k)[1] = addr(pair[1])
                setattr(b, n, int(buffers[n]))
        self._buffers = buffers
        h = ctypes.c_void_p()
        self.handle = None
        _check(load().pa_graph_create(ctypes.byref(self._descs[0]), ctypes.byref(self._shape), ctypes.byref(b),
                                      ctypes.byref(h)), "pa_graph_create")
        self.handle = h.value
        self._step = load().pa_graph_step
        self._turn = 0

    def step(self, num_reqs: int, stream=None, num_common_prefix_blocks: int = 0):
        """Plan the step now in the host arrays (set ``turn``) and launch the
        next graph (num_common_prefix_blocks > 0: the cascade route)."""
        d = self._descs[self._turn]
        d.num_reqs = num_reqs
        d.num_common_prefix_blocks = num_common_prefix_blocks
        _check(self._step(self.handle, ctypes.byref(d), _stream(stream)), "pa_graph_step")
        self._turn = 1 - self._turn

    @property
    def turn(self) -> int:
        """Graph (and host set / I/O buffers) the next step uses."""
        return int(load().pa_graph_turn(self.handle))

    def wait(self, turn: int):
        _check(load().pa_graph_wait(self.handle, int(turn)), "pa_graph_wait")

    def workspace_ptr(self) -> int:
        return int(load().pa_graph_workspace(self.handle))

    def slot_mapping_ptr(self) -> int:
        return int(load().pa_graph_slot_mapping(self.handle))

    def destroy(self):
        if self.handle:
            load().pa_graph_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass
