"""ctypes binding of liblstream.so: the C ABI of include/ls_api.h and include/ls_kernels.h
under the same names. It only marshals arguments (torch tensors and numpy
arrays to pointers, Python lists to C arrays); all work happens in the library.

Negative status codes raise ``LsError`` carrying the context's ``ls_last_error``;
warnings (positive codes) are returned.
"""
from __future__ import annotations

import ctypes as C
import os
import struct
import sys

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "liblstream.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()' "
        "or python host_offloaded_weight_gb300/build.py). There is no fallback path.")
_lib = C.CDLL(LIB_PATH)

# ------------------------------------------------------------------ constants
LS_PARAMS_VERSION = 1
LS_OK, LS_WARN_MANDATORY_SLOT, LS_WARN_SYNC_FALLBACK = 0, 1, 2
LS_ERR_INVALID_ARG, LS_ERR_VERSION, LS_ERR_OOM = -1, -2, -3
LS_ERR_HANDOFF_TIMEOUT, LS_ERR_CUDA, LS_ERR_STATE, LS_ERR_UNSUPPORTED, LS_ERR_BOUNDS = -4, -5, -6, -7, -8
LS_KIND_LINEAR_GELU_F32, LS_KIND_FFN_GELU_BF16, LS_KIND_FFN_GELU_SHARED_BF16 = 0, 1, 2
LS_KIND_SWIGLU_BF16, LS_KIND_MOE_SWIGLU_BF16 = 3, 4
LS_DTYPE_F32, LS_DTYPE_BF16 = 0, 1
LS_EV_SHARED_LOAD, LS_EV_LOAD_RESIDENT, LS_EV_LOAD_SYNC, LS_EV_PREFETCH, LS_EV_ACTIVATE, LS_EV_EVICT = range(6)
LS_COPY_AUTO, LS_COPY_KERNEL, LS_COPY_ENGINE = 0, 1, 2
LSK_EPI_STORE, LSK_EPI_BIAS_GELU, LSK_EPI_BIAS_RESID, LSK_EPI_SWIGLU, LSK_EPI_RESID, LSK_EPI_SCALE_F32 = range(6)

ALLOC_FN = C.CFUNCTYPE(C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p)
FREE_FN = C.CFUNCTYPE(None, C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p)


class ls_params(C.Structure):
    _fields_ = [("struct_size", C.c_uint32), ("version", C.c_uint32),
                ("prefetch_depth", C.c_int32), ("resident_layers", C.c_int32),
                ("max_vram_bytes", C.c_int64), ("use_pool", C.c_int32),
                ("wait_limit_ms", C.c_int32), ("copy_path", C.c_int32), ("copy_ctas", C.c_int32),
                ("reserve_sms", C.c_int32), ("device", C.c_int32),
                ("alloc_fn", ALLOC_FN), ("free_fn", FREE_FN), ("alloc_user", C.c_void_p),
                ("test_alloc_cap_bytes", C.c_int64), ("test_fail_async", C.c_int32),
                ("test_drop_publish", C.c_int32), ("kernel_timing", C.c_int32),
                ("cross_run_prefetch", C.c_int32), ("expert_cache_bytes", C.c_int64),
                ("debug_checks", C.c_int32), ("test_corrupt_canary", C.c_int32),
                ("test_kernel_copy_stride", C.c_int32)]


class ls_tensor_desc(C.Structure):
    _fields_ = [("host_ptr", C.c_void_p), ("bytes", C.c_uint64), ("dtype", C.c_int32),
                ("ndim", C.c_int32), ("shape", C.c_int64 * 2)]


class ls_segment_desc(C.Structure):
    _fields_ = [("kind", C.c_int32), ("n_tensors", C.c_int32),
                ("tensors", C.POINTER(ls_tensor_desc))]


class ls_shared_ref(C.Structure):
    _fields_ = [("segment", C.c_int32), ("tensor_index", C.c_int32), ("shared_id", C.c_int32)]


class ls_moe_routing(C.Structure):
    _fields_ = [("logits", C.c_void_p), ("top_k", C.c_int32)]


class lsk_moe_experts(C.Structure):
    _fields_ = [("mxfp4", C.c_int32), ("reserved", C.c_int32), ("gate", C.c_void_p), ("up", C.c_void_p),
                ("down", C.c_void_p), ("gate_stride", C.c_int64), ("down_stride", C.c_int64),
                ("gate_scales", C.c_void_p), ("up_scales", C.c_void_p), ("down_scales", C.c_void_p),
                ("gate_scale_stride", C.c_int64), ("down_scale_stride", C.c_int64)]


class lsk_lora(C.Structure):
    _fields_ = [("n", C.c_int32), ("rank", C.c_int32), ("down", C.c_void_p), ("up", C.c_void_p), ("up2", C.c_void_p),
                ("scale", C.c_void_p), ("down_stride", C.c_int64), ("up_stride", C.c_int64)]


class ls_kernel_time(C.Structure):
    _fields_ = [("name", C.c_char * 32), ("launches", C.c_int64), ("total_ms", C.c_double)]


class ls_trace_event(C.Structure):
    _fields_ = [("name", C.c_char * 32), ("stream", C.c_int32), ("segment", C.c_int32),
                ("start_ms", C.c_double), ("end_ms", C.c_double)]


class ls_sched_event(C.Structure):
    _fields_ = [("run", C.c_int32), ("step", C.c_int32), ("kind", C.c_int32),
                ("segment", C.c_int32), ("slot", C.c_int32), ("reserved", C.c_int32),
                ("bytes", C.c_int64)]


class ls_stats(C.Structure):
    _fields_ = [("struct_size", C.c_uint32), ("n_segments", C.c_int32), ("residents", C.c_int32),
                ("depth", C.c_int32), ("ring_slots", C.c_int32), ("pool_slots", C.c_int32),
                ("warnings", C.c_int32), ("copy_path", C.c_int32), ("slot_bytes", C.c_int64),
                ("shared_bytes", C.c_int64), ("pool_bytes", C.c_int64), ("runs", C.c_int64),
                ("prefetch_queued", C.c_int64), ("prefetch_activated", C.c_int64),
                ("sync_loads", C.c_int64), ("resident_loads", C.c_int64),
                ("shared_loads", C.c_int64), ("evictions", C.c_int64),
                ("sync_fallbacks", C.c_int64), ("pool_degradations", C.c_int64),
                ("bytes_loaded", C.c_int64), ("copy_kernel_gbs", C.c_double),
                ("copy_engine_gbs", C.c_double), ("graph_captures", C.c_int64),
                ("graph_replays", C.c_int64), ("expert_cache_hits", C.c_int64),
                ("expert_host_loads", C.c_int64), ("debug_violations", C.c_int64),
                ("kernel_copy_segments", C.c_int64)]


_P = C.c_void_p
_I32, _I64, _U32, _U64 = C.c_int32, C.c_int64, C.c_uint32, C.c_uint64
_sig = {
    "ls_params_init": (None, [C.POINTER(ls_params)]),
    "ls_ctx_create": (_I32, [C.POINTER(ls_params), C.POINTER(_P)]),
    "ls_register_segments": (_I32, [_P, C.POINTER(ls_segment_desc), _I32, C.POINTER(ls_shared_ref), _I32]),
    "ls_run": (_I32, [_P, _P, _P, _I64, _P, C.POINTER(ls_moe_routing)]),
    "ls_run_host": (_I32, [_P, _P, _P, _I64, C.POINTER(ls_moe_routing)]),
    "ls_run_host_async": (_I32, [_P, _P, _P, _I64, C.POINTER(ls_moe_routing)]),
    "ls_run_async": (_I32, [_P, _P, _P, _I64, _P, C.POINTER(ls_moe_routing)]),
    "ls_sync": (_I32, [_P]),
    "ls_get_schedule": (_I32, [_P, C.POINTER(ls_sched_event), _I64, C.POINTER(_I64)]),
    "ls_get_stats": (_I32, [_P, C.POINTER(ls_stats)]),
    "ls_set_kernel_timing": (_I32, [_P, _I32]),
    "ls_replan": (_I32, [_P, _I32, _I32, _I64]),
    "ls_run_graph": (_I32, [_P, _P, _P, _I64, _P]),
    "ls_simulate_script": (_I32, [C.POINTER(ls_params), C.POINTER(_I64), _I32, C.POINTER(_I64),
                                  C.POINTER(_I32), _I32, C.POINTER(_I64), _I32, C.POINTER(ls_sched_event),
                                  _I64, C.POINTER(_I64), C.POINTER(ls_stats), C.POINTER(_I32)]),
    "ls_get_kernel_times": (_I32, [_P, C.POINTER(ls_kernel_time), _I32, C.POINTER(_I32), _I32]),
    "ls_get_trace": (_I32, [_P, C.POINTER(ls_trace_event), _I64, C.POINTER(_I64)]),
    "ls_ctx_destroy": (None, [_P]),
    "ls_status_string": (C.c_char_p, [_I32]),
    "ls_last_error": (C.c_char_p, [_P]),
    "ls_simulate": (_I32, [C.POINTER(ls_params), C.POINTER(_I64), _I32, C.POINTER(_I64),
                           C.POINTER(_I32), _I32, _I32, C.POINTER(_I64), C.POINTER(ls_sched_event),
                           _I64, C.POINTER(_I64), C.POINTER(ls_stats), C.POINTER(_I32)]),
    "lsk_num_sms": (_I32, []),
    "lsk_gemm_tile_n": (_I32, [_I32, _I32, _I32]),
    "lsk_device_error": (_U32, []),
    "lsk_copy_h2slot": (_I32, [_P, _P, _U64, _I32, _P, _P, _U32, _P]),
    "lsk_wait_ready": (_I32, [_P, _U32, _I32, _P, _I32, _P]),
    "lsk_copy_h2slot_static": (_I32, [_P, C.POINTER(_P), C.POINTER(_U64), C.POINTER(_U64), _I32, _I32, _P,
                                      _U32, _P]),
    "lsk_gemm_bf16": (_I32, [_I32, _P, _P, _I64, _I32, _P, _P, _I32, _P, _P, _I32, _I32, _I32, _I32, _P]),
    "lsk_gemm_grouped_bf16": (_I32, [_I32, _P, _P, _I64, _I32, _I32, _I32, _P, _I32, _P, _P, _P,
                                     _I32, _I32, _I32, _I32, _P]),
    "lsk_linear_gelu_f32": (_I32, [_P, _P, _P, _P, _I32, _I32, _I32, _P]),
    "lsk_moe_route": (_I32, [_P, _I32, _I32, _I32, _I32, _P, _P, _P]),
    "lsk_moe_group": (_I32, [_P, _I32, _I32, _I32, _I32, _P, _P, _P, _P]),
    "lsk_moe_gather": (_I32, [_P, _P, _I32, _I32, _I32, _P, _P]),
    "lsk_moe_combine": (_I32, [_P, _I32, _P, _I32, _I32, _I32, _P, _P, _P]),
    "lsk_moe_check": (_I32, [_P, _P, _P, _I32, _I32, _I32, _I32, _P, _P]),
    "lsk_moe_group_masked": (_I32, [_P, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _P]),
    "lsk_moe_rows_copy": (_I32, [_P, _P, _P, _P, _I32, _I32, _P, _P, _U32, _I32, _P]),
    "lsk_mxfp4_code_pitch": (_I64, [_I32]),
    "lsk_mxfp4_scale_pitch": (_I64, [_I32]),
    "lsk_mxfp4_quantize": (_I32, [_P, _I32, _I64, _I32, _I64, _P, _P, _P]),
    "lsk_mxfp4_dequantize": (_I32, [_P, _P, _I64, _I32, _P, _I32, _I64, _P]),
    "lsk_gemm_mxfp4": (_I32, [_P, _P, _P, _P, _P, _I32, _I32, _I32, _I32, _P]),
    "lsk_gemm_bf16_mxfp4": (_I32, [_P, _I64, _P, _P, _P, _I32, _I32, _I32, _I32, _P]),
    "lsk_moe_few": (_I32, [_P, _P, _P, _P, _I32, _I32, _I32, _I32, _I32, _P, _P, _P]),
    "lsk_gemm_lora_bf16": (_I32, [_I32, _P, _P, _I64, _I32, _P, _P, _P, _P, _I32, _P, _P, _I32, _I32, _I32, _P]),
    "lsk_gemm_grouped_bf16_mxfp4": (_I32, [_I32, _P, _I64, _P, _P, _P, _P, _I64, _I64, _P, _I32, _P, _P, _I32, _P, _I32, _I32, _I32, _P]),
    "ls_helper_share": (C.c_double, [_I64]),
    "ls_host_alloc": (_I32, [_U64, C.POINTER(_P)]),
    "ls_host_free": (_I32, [_P]),
    "ls_helper_split": (_I32, [_P, _I32, C.c_double, _P]),
}
for _name, (_res, _args) in _sig.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args

EXPORTED = tuple(_sig)


class LsError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{ls_status_string(status)} ({status}): {msg}")
        self.status = status


def ls_status_string(s: int) -> str:
    return _lib.ls_status_string(int(s)).decode()


def _check(status: int, ctx=None) -> int:
    if status < 0:
        msg = _lib.ls_last_error(ctx.handle if isinstance(ctx, Ctx) else ctx).decode() if ctx else ""
        raise LsError(status, msg)
    return status


def _ptr(t) -> int:
    """Address of a torch tensor, numpy array or raw int pointer (None -> 0)."""
    if t is None:
        return 0
    try:
        return t.data_ptr()
    except AttributeError:
        pass
    if isinstance(t, int):
        return t
    if hasattr(t, "ctypes"):
        return t.ctypes.data
    raise TypeError(f"cannot take the address of {type(t)}")


_current_stream = None


def _bind_current_stream():
    """The raw handle of torch's current stream, without building a Stream object (2.7 us of a
    5 us call on the GB300's host); torch.cuda.current_stream() where torch has no such function."""
    global _current_stream
    import torch
    raw, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
    if raw is None or device is None:
        _current_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
    else:
        torch.cuda.init()
        _current_stream = lambda: raw(device())  # noqa: E731


def _stream(stream) -> int:
    if stream is None:
        if _current_stream is None:
            _bind_current_stream()
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


class Ctx:
    """A context handle plus references to the host buffers it reads."""

    def __init__(self, handle: int):
        self.handle = handle
        self.keep = []

    def __bool__(self):
        return bool(self.handle)


# ------------------------------------------------------------------ ls_api.h
def ls_params_init(**fields) -> ls_params:
    p = ls_params()
    _lib.ls_params_init(C.byref(p))
    for k, v in fields.items():
        setattr(p, k, v)
    return p


def ls_ctx_create(params: ls_params) -> Ctx:
    h = _P()
    _check(_lib.ls_ctx_create(C.byref(params), C.byref(h)))
    return Ctx(h.value)


def _dtype_code(t) -> int:
    name = str(getattr(t, "dtype", ""))
    if "float32" in name:
        return LS_DTYPE_F32
    if "bfloat16" in name or "uint16" in name:
        return LS_DTYPE_BF16
    raise TypeError(f"unsupported tensor dtype {name}")


def _nbytes(t) -> int:
    if hasattr(t, "nbytes"):
        return int(t.nbytes)
    return t.numel() * t.element_size()


def ls_register_segments(ctx: Ctx, segments, shared_map=()) -> int:
    """segments: list of (kind, [host tensors]) — torch CPU tensors (pinned or
    not) or numpy arrays; bf16 may be given as uint16 bit patterns.
    shared_map: list of (segment, tensor_index, shared_id)."""
    segs = (ls_segment_desc * len(segments))()
    for i, (kind, tensors) in enumerate(segments):
        arr = (ls_tensor_desc * len(tensors))()
        for j, t in enumerate(tensors):
            shape = tuple(t.shape)
            arr[j].host_ptr = _ptr(t)
            arr[j].bytes = _nbytes(t)
            arr[j].dtype = _dtype_code(t)
            arr[j].ndim = len(shape)
            for d, v in enumerate(shape[:2]):
                arr[j].shape[d] = v
            ctx.keep.append(t)
        ctx.keep.append(arr)
        segs[i].kind = kind
        segs[i].n_tensors = len(tensors)
        segs[i].tensors = arr
    sm = (ls_shared_ref * max(1, len(shared_map)))()
    for i, (s, ti, sid) in enumerate(shared_map):
        sm[i].segment, sm[i].tensor_index, sm[i].shared_id = s, ti, sid
    return _check(_lib.ls_register_segments(ctx.handle, segs, len(segments), sm, len(shared_map)), ctx)


def _routing(logits, top_k):
    if logits is None:
        return None
    r = ls_moe_routing()
    r.logits = _ptr(logits)
    r.top_k = top_k
    return r


def ls_run(ctx: Ctx, x, y, tokens: int, stream=None, logits=None, top_k: int = 0) -> int:
    """One streamed pass on device tensors (stream: torch stream, raw handle or None = current)."""
    r = _routing(logits, top_k)
    return _check(_lib.ls_run(ctx.handle, _ptr(x), _ptr(y), int(tokens), _stream(stream),
                              C.byref(r) if r is not None else None), ctx)


def ls_run_async(ctx: Ctx, x, y, tokens: int, stream=None, logits=None, top_k: int = 0) -> int:
    """Queue one pass without waiting for it; ls_sync reports device errors."""
    r = _routing(logits, top_k)
    return _check(_lib.ls_run_async(ctx.handle, _ptr(x), _ptr(y), int(tokens), _stream(stream),
                                    C.byref(r) if r is not None else None), ctx)


def ls_sync(ctx: Ctx) -> int:
    return _check(_lib.ls_sync(ctx.handle), ctx)


def ls_run_host(ctx: Ctx, x_host, y_host, tokens: int, logits_host=None, top_k: int = 0) -> int:
    r = _routing(logits_host, top_k)
    return _check(_lib.ls_run_host(ctx.handle, _ptr(x_host), _ptr(y_host), int(tokens),
                                   C.byref(r) if r is not None else None), ctx)


def ls_run_host_async(ctx: Ctx, x_host, y_host, tokens: int, logits_host=None, top_k: int = 0) -> int:
    """ls_run_host queued on the context's own stream; y_host is valid after ls_sync."""
    r = _routing(logits_host, top_k)
    return _check(_lib.ls_run_host_async(ctx.handle, _ptr(x_host), _ptr(y_host), int(tokens),
                                         C.byref(r) if r is not None else None), ctx)


def _events(buf, n):
    return [(e.run, e.step, e.kind, e.segment, e.slot, e.bytes) for e in buf[:n]]


def ls_get_schedule(ctx: Ctx) -> list:
    n = _I64()
    _check(_lib.ls_get_schedule(ctx.handle, None, 0, C.byref(n)), ctx)
    buf = (ls_sched_event * max(1, n.value))()
    _check(_lib.ls_get_schedule(ctx.handle, buf, n.value, C.byref(n)), ctx)
    return _events(buf, n.value)


def _stats_dict(s: ls_stats) -> dict:
    return {name: getattr(s, name) for name, _ in ls_stats._fields_}


def ls_get_stats(ctx: Ctx) -> dict:
    s = ls_stats()
    s.struct_size = C.sizeof(ls_stats)
    _check(_lib.ls_get_stats(ctx.handle, C.byref(s)), ctx)
    return _stats_dict(s)


def ls_run_graph(ctx: Ctx, x, y, tokens: int, stream=None) -> int:
    """One pass issued as a CUDA graph replay once the pass is steady (see include/ls_api.h)."""
    return _check(_lib.ls_run_graph(ctx.handle, _ptr(x), _ptr(y), tokens, _stream(stream)), ctx)


def ls_replan(ctx: Ctx, prefetch_depth: int, resident_layers: int, max_vram_bytes: int) -> int:
    """New streaming controls for the next run (see include/ls_api.h)."""
    return _check(_lib.ls_replan(ctx.handle, prefetch_depth, resident_layers, max_vram_bytes), ctx)


def ls_set_kernel_timing(ctx: Ctx, mode: int) -> int:
    return _check(_lib.ls_set_kernel_timing(ctx.handle, mode), ctx)


def ls_get_kernel_times(ctx: Ctx, reset: bool = False) -> dict:
    """{kernel class: (launches, total_ms)} accumulated while kernel_timing is on."""
    n = _I32()
    _check(_lib.ls_get_kernel_times(ctx.handle, None, 0, C.byref(n), 0), ctx)
    buf = (ls_kernel_time * max(1, n.value))()
    _check(_lib.ls_get_kernel_times(ctx.handle, buf, n.value, C.byref(n), int(reset)), ctx)
    return {buf[i].name.decode(): (buf[i].launches, buf[i].total_ms) for i in range(n.value)}


def ls_get_trace(ctx: Ctx) -> list:
    """[(name, stream, segment, start_ms, end_ms)] of the passes the last ls_sync completed."""
    n = _I64()
    _check(_lib.ls_get_trace(ctx.handle, None, 0, C.byref(n)), ctx)
    buf = (ls_trace_event * max(1, n.value))()
    _check(_lib.ls_get_trace(ctx.handle, buf, n.value, C.byref(n)), ctx)
    return [(b.name.decode(), b.stream, b.segment, b.start_ms, b.end_ms) for b in buf[:n.value]]


def ls_ctx_destroy(ctx: Ctx) -> None:
    if ctx and ctx.handle:
        _lib.ls_ctx_destroy(ctx.handle)
        ctx.handle = 0
        ctx.keep.clear()


def ls_last_error(ctx: Ctx) -> str:
    return _lib.ls_last_error(ctx.handle).decode()


def ls_simulate(params: ls_params, seg_slot_bytes, shared=(), runs: int = 1, load_bytes=None):
    """Returns (status, events, stats, run_status) from the library's scheduler
    run without a GPU. shared: [(shared_id, bytes)]; load_bytes: [runs][n] or None."""
    n = len(seg_slot_bytes)
    seg = (_I64 * n)(*seg_slot_bytes)
    sb = (_I64 * max(1, len(shared)))(*[b for _, b in shared])
    sid = (_I32 * max(1, len(shared)))(*[i for i, _ in shared])
    lb = None
    if load_bytes is not None:
        flat = [int(v) for row in load_bytes for v in row]
        lb = (_I64 * len(flat))(*flat)
    total = _I64()
    st = ls_stats()
    st.struct_size = C.sizeof(ls_stats)
    rs = (_I32 * max(1, runs))()
    status = _lib.ls_simulate(C.byref(params), seg, n, sb, sid, len(shared), runs, lb, None, 0,
                              C.byref(total), C.byref(st), rs)
    buf = (ls_sched_event * max(1, total.value))()
    status = _lib.ls_simulate(C.byref(params), seg, n, sb, sid, len(shared), runs, lb, buf,
                              total.value, C.byref(total), C.byref(st), rs)
    return status, _events(buf, total.value), _stats_dict(st), list(rs[:runs])


def ls_simulate_script(params: ls_params, seg_slot_bytes, script, shared=()):
    """ls_simulate along a script of ("run",) and ("replan", depth, resident, max_vram)
    steps. Returns (status, events, stats, step_status)."""
    n = len(seg_slot_bytes)
    seg = (_I64 * n)(*seg_slot_bytes)
    sb = (_I64 * max(1, len(shared)))(*[b for _, b in shared])
    sid = (_I32 * max(1, len(shared)))(*[i for i, _ in shared])
    flat = []
    for step in script:
        flat += [0, 0, 0, 0] if step[0] == "run" else [1, int(step[1]), int(step[2]), int(step[3])]
    sc = (_I64 * max(1, len(flat)))(*flat)
    total = _I64()
    st = ls_stats()
    st.struct_size = C.sizeof(ls_stats)
    ss = (_I32 * max(1, len(script)))(*([1 << 30] * max(1, len(script))))
    status = _lib.ls_simulate_script(C.byref(params), seg, n, sb, sid, len(shared), sc, len(script), None, 0,
                                     C.byref(total), C.byref(st), ss)
    buf = (ls_sched_event * max(1, total.value))()
    ss = (_I32 * max(1, len(script)))(*([1 << 30] * max(1, len(script))))
    status = _lib.ls_simulate_script(C.byref(params), seg, n, sb, sid, len(shared), sc, len(script), buf,
                                     total.value, C.byref(total), C.byref(st), ss)
    steps = [v for v in ss[:len(script)] if v != 1 << 30]
    return status, _events(buf, total.value), _stats_dict(st), steps


# ------------------------------------------------------------------ ls_kernels.h
def lsk_num_sms() -> int:
    return _lib.lsk_num_sms()


def lsk_gemm_tile_n(epilogue: int, M: int, N: int) -> int:
    """Output columns of one tile of lsk_gemm_bf16 for an M x N output on this device."""
    return _lib.lsk_gemm_tile_n(epilogue, M, N)


def lsk_device_error() -> int:
    return _lib.lsk_device_error()


def lsk_copy_h2slot(dst, src_host, nbytes: int, ctas: int, ready, ticket, epoch: int, stream=None) -> int:
    return _check(_lib.lsk_copy_h2slot(_ptr(dst), _ptr(src_host), int(nbytes), ctas, _ptr(ready),
                                       _ptr(ticket), epoch, _stream(stream)))


LSK_STATIC_MAX_RANGES = 64


def lsk_copy_h2slot_static(dst, srcs, sizes, dst_offsets, ctas: int, ready, epoch: int, stream=None) -> int:
    """The copy and publish of lsk_copy_h2slot for up to 64 pinned host ranges,
    without allocating device memory (its scratch is a fixed array in the library)."""
    n = len(srcs)
    src_arr = (_P * max(1, n))(*[_ptr(s) for s in srcs])
    sz = (_U64 * max(1, n))(*[int(b) for b in sizes])
    off = (_U64 * max(1, n))(*[int(o) for o in dst_offsets])
    return _check(_lib.lsk_copy_h2slot_static(_ptr(dst), src_arr, sz, off, n, ctas, _ptr(ready), epoch,
                                              _stream(stream)))


def lsk_wait_ready(ready, epoch: int, limit_ms: int, err_host, slot: int = 0, stream=None) -> int:
    return _check(_lib.lsk_wait_ready(_ptr(ready), epoch, limit_ms, _ptr(err_host), slot, _stream(stream)))


def lsk_gemm_bf16(epilogue: int, A, B, C_out, M: int, N: int, K: int, bias=None, resid=None,
                  b_rows: int | None = None, b2_row_off: int = 0, max_ctas: int = 0, stream=None,
                  C32=None) -> int:
    rows = b_rows if b_rows is not None else B.shape[0]
    rf32 = int(resid is not None and "float32" in str(getattr(resid, "dtype", "")))
    return _check(_lib.lsk_gemm_bf16(epilogue, _ptr(A), _ptr(B), rows, b2_row_off, _ptr(bias),
                                     _ptr(resid), rf32, _ptr(C_out), _ptr(C32), M, N, K, max_ctas,
                                     _stream(stream)))


def lsk_gemm_grouped_bf16(epilogue: int, A, B, b_rows: int, b_base_row: int, b_group_stride_rows: int,
                          b2_row_off: int, group_bounds, n_groups: int, C_out, M: int, N: int, K: int,
                          row_table=None, row_weight=None, max_ctas: int = 0, stream=None) -> int:
    return _check(_lib.lsk_gemm_grouped_bf16(
        epilogue, _ptr(A), _ptr(B), b_rows, b_base_row, b_group_stride_rows, b2_row_off,
        _ptr(group_bounds), n_groups, _ptr(row_table), _ptr(row_weight), _ptr(C_out), M, N, K,
        max_ctas, _stream(stream)))


def lsk_linear_gelu_f32(x, w, b, y, T: int, H: int, F: int, stream=None) -> int:
    return _check(_lib.lsk_linear_gelu_f32(_ptr(x), _ptr(w), _ptr(b), _ptr(y), T, H, F, _stream(stream)))


def lsk_moe_route(logits, n_layers, T, E, k, sel, weight, stream=None) -> int:
    return _check(_lib.lsk_moe_route(_ptr(logits), n_layers, T, E, k, _ptr(sel), _ptr(weight),
                                     _stream(stream)))


def lsk_moe_group(sel, n_layers, T, E, k, row_table, group_bounds, expert_used=None, stream=None) -> int:
    return _check(_lib.lsk_moe_group(_ptr(sel), n_layers, T, E, k, _ptr(row_table), _ptr(group_bounds),
                                     _ptr(expert_used), _stream(stream)))


def lsk_moe_gather(x, row_table, rows, k, H, x_sorted, stream=None) -> int:
    return _check(_lib.lsk_moe_gather(_ptr(x), _ptr(row_table), rows, k, H, _ptr(x_sorted), _stream(stream)))


def lsk_moe_check(sel, row_table, group_bounds, n_layers: int, T: int, k: int, E: int, err_host,
                  stream=None) -> int:
    return _check(_lib.lsk_moe_check(_ptr(sel), _ptr(row_table), _ptr(group_bounds), n_layers, T, k, E,
                                     _ptr(err_host), _stream(stream)))


def lsk_moe_group_masked(sel, n_layers, T, E, k, expert_mask, row_table, group_bounds, expert_used=None,
                         stream=None) -> int:
    return _check(_lib.lsk_moe_group_masked(_ptr(sel), n_layers, T, E, k, _ptr(expert_mask), _ptr(row_table),
                                            _ptr(group_bounds), _ptr(expert_used), _stream(stream)))


def lsk_moe_rows_copy(src, dst, rows: int, H: int, src_table=None, dst_table=None, ready=None, ticket=None,
                      epoch: int = 0, ctas: int = 0, stream=None) -> int:
    return _check(_lib.lsk_moe_rows_copy(_ptr(src), _ptr(src_table), _ptr(dst), _ptr(dst_table), rows, H,
                                         _ptr(ready), _ptr(ticket), epoch, ctas, _stream(stream)))


def ls_host_alloc(nbytes: int) -> int:
    """Pinned, device-mapped host memory of nbytes bytes (address as an int)."""
    p = _P()
    _check(_lib.ls_host_alloc(nbytes, C.byref(p)))
    return p.value


def ls_host_free(ptr: int) -> None:
    _check(_lib.ls_host_free(ptr))


def ls_helper_share(tokens: int) -> float:
    return float(_lib.ls_helper_share(tokens))


def ls_helper_split(routed, share: float):
    """routed: uint8 numpy array [E] (nonzero = routed) -> the helper's mask, uint8 [E]."""
    import numpy as np
    r = np.ascontiguousarray(routed, dtype=np.uint8)
    out = np.zeros_like(r)
    _check(_lib.ls_helper_split(_ptr(r), r.size, share, _ptr(out)))
    return out


def lsk_moe_combine(x, y, T, k, H, out, out32=None, stream=None) -> int:
    xf32 = int("float32" in str(getattr(x, "dtype", "")))
    return _check(_lib.lsk_moe_combine(_ptr(x), xf32, _ptr(y), T, k, H, _ptr(out), _ptr(out32), _stream(stream)))


# ------------------------------------------------------------------ MXFP4
_f32_of = {None: 0}  # a tensor's dtype -> whether it is float32, as far as they have been met


def _is_f32(t) -> int:
    """1 for float32, 0 for bf16 and for raw addresses; other types are a TypeError."""
    d = getattr(t, "dtype", None)
    try:
        return _f32_of[d]
    except KeyError:
        _f32_of[d] = int(_dtype_code(t) == LS_DTYPE_F32)
        return _f32_of[d]


def lsk_mxfp4_code_pitch(K: int) -> int:
    """Bytes of a row of K 4-bit codes."""
    return _lib.lsk_mxfp4_code_pitch(K)


def lsk_mxfp4_scale_pitch(K: int) -> int:
    """Bytes of a row's block scales."""
    return _lib.lsk_mxfp4_scale_pitch(K)


def _dense(t, what: str):
    f = getattr(t, "is_contiguous", None)
    if not (f() if f is not None else t.flags.c_contiguous):
        raise ValueError(f"{what} is not dense")


def _values(t, f32: int, what: str) -> int:
    """Address of a dense bf16 (f32 = 0) or float32 (1) tensor; raw addresses and None pass."""
    if getattr(t, "dtype", None) is not None:
        if _is_f32(t) != f32:
            raise TypeError(f"{what} has to be {'float32' if f32 else 'bf16'}, not {t.dtype}")
        _dense(t, what)
    return _ptr(t)


def _rows(t, ld, what: str):
    """A matrix's rows: dense, or ld elements apart and dense in themselves."""
    if getattr(t, "dtype", None) is None:
        return
    if ld is None:
        _dense(t, what)
    elif hasattr(t, "stride") and t.dim() and t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"the rows of {what} are not dense")


def _bytes(t, what: str) -> int:
    """Address of a dense tensor of codes or scales (a byte each)."""
    if getattr(t, "dtype", None) is not None:
        if t.itemsize != 1:
            raise TypeError(f"{what} has to be bytes, not {t.dtype}")
        _dense(t, what)
    return _ptr(t)


def _expert_rows(t, what: str):
    """Experts may lie apart; the rows of each are dense."""
    if not t.is_contiguous():
        shape, stride = t.shape, t.stride()
        if len(shape) < 2 or (stride[-1] != 1 and shape[-1] > 1) or (stride[-2] != shape[-1] and shape[-2] > 1):
            raise ValueError(f"an expert's rows of {what} are not dense")


# The usual arguments (torch tensors of the right types, dense) are recognised in few steps, since a check of each by the
# functions above would cost a one-token layer 2 us of its call; all others take those functions.
_BF16 = _F32 = _U8 = _INT32 = None


def _bind_types():
    global _BF16, _F32, _U8, _INT32
    torch = sys.modules.get("torch")
    if torch is not None:
        _BF16, _F32, _U8, _INT32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


def _conversion(values, ld, codes, scales, what: str):
    """Addresses of a conversion's matrix, codes and scales."""
    try:
        usual = (codes.dtype is _U8 and scales.dtype is _U8 and codes.is_contiguous() and scales.is_contiguous()
                 and (values.is_contiguous() if ld is None else values.stride(-1) == 1))
    except (AttributeError, IndexError, TypeError):
        usual = False
    if usual:
        return values.data_ptr(), codes.data_ptr(), scales.data_ptr()
    _bind_types()
    _rows(values, ld, what)
    return _ptr(values), _bytes(codes, "codes"), _bytes(scales, "scales")


def lsk_mxfp4_quantize(src, rows: int, K: int, codes, scales, ld: int | None = None, stream=None) -> int:
    """src [rows, K] bf16 or float32, ld elements between rows (None = K, dense)."""
    v, c, s = _conversion(src, ld, codes, scales, "src")
    return _check(_lib.lsk_mxfp4_quantize(v, _is_f32(src), rows, K, K if ld is None else ld, c, s, _stream(stream)))


def lsk_mxfp4_dequantize(codes, scales, rows: int, K: int, dst, ld: int | None = None, stream=None) -> int:
    """dst [rows, K] bf16 or float32, ld elements between rows (None = K, dense)."""
    v, c, s = _conversion(dst, ld, codes, scales, "dst")
    return _check(_lib.lsk_mxfp4_dequantize(c, s, rows, K, v, _is_f32(dst), K if ld is None else ld, _stream(stream)))


def lsk_gemm_mxfp4(A_codes, A_scales, B_codes, B_scales, C_out, M: int, N: int, K: int, stream=None) -> int:
    """C_out [M, N] bf16 or float32, dense."""
    try:
        f32 = 1 if C_out.dtype is _F32 else 0
        usual = ((f32 or C_out.dtype is _BF16) and A_codes.dtype is _U8 and A_scales.dtype is _U8
                 and B_codes.dtype is _U8 and B_scales.dtype is _U8 and A_codes.is_contiguous() and A_scales.is_contiguous()
                 and B_codes.is_contiguous() and B_scales.is_contiguous() and C_out.is_contiguous())
    except AttributeError:
        usual = False
    if usual:
        ac, as_, bc, bs, c = A_codes.data_ptr(), A_scales.data_ptr(), B_codes.data_ptr(), B_scales.data_ptr(), C_out.data_ptr()
    else:
        _bind_types()
        f32 = _is_f32(C_out)
        ac, as_ = _bytes(A_codes, "A_codes"), _bytes(A_scales, "A_scales")
        bc, bs, c = _bytes(B_codes, "B_codes"), _bytes(B_scales, "B_scales"), _values(C_out, f32, "C_out")
    return _check(_lib.lsk_gemm_mxfp4(ac, as_, bc, bs, c, f32, M, N, K, _stream(stream)))


def lsk_gemm_bf16_mxfp4(A, B_codes, B_scales, C_out, M: int, N: int, K: int, lda: int | None = None,
                        stream=None) -> int:
    """A [M, K] bf16, lda elements between rows (None = K, dense); C_out [M, N] bf16 or float32, dense."""
    try:
        f32 = 1 if C_out.dtype is _F32 else 0
        usual = ((f32 or C_out.dtype is _BF16) and A.dtype is _BF16 and lda is None and A.is_contiguous()
                 and B_codes.dtype is _U8 and B_scales.dtype is _U8 and B_codes.is_contiguous()
                 and B_scales.is_contiguous() and C_out.is_contiguous())
    except AttributeError:
        usual = False
    if usual:
        lda, a, b, bs, c = K, A.data_ptr(), B_codes.data_ptr(), B_scales.data_ptr(), C_out.data_ptr()
    else:
        _bind_types()
        if _is_f32(A):
            raise TypeError("A has to be bf16, not float32")
        _rows(A, lda, "A")
        lda, f32 = K if lda is None else lda, _is_f32(C_out)
        a, b, bs, c = _ptr(A), _bytes(B_codes, "B_codes"), _bytes(B_scales, "B_scales"), _values(C_out, f32, "C_out")
    return _check(_lib.lsk_gemm_bf16_mxfp4(a, lda, b, bs, c, f32, M, N, K, _stream(stream)))


_experts = struct.Struct("@2i10q").pack   # lsk_moe_experts, as bytes: a third of the time that the ctypes structure takes


def lsk_moe_few(x, logits, gate, up, down, T: int, E: int, k: int, H: int, F: int, out, gate_scales=None,
                up_scales=None, down_scales=None, resid=None, out32=None, stream=None) -> int:
    """One MoE layer for T <= 64 tokens. x and out [T, H] bf16, logits [T, E], resid and out32 [T, H] float32, all dense.
    gate, up [E, F, H] and down [E, H, F] bf16, or MXFP4 codes [E, rows, code pitch] with their scales
    [E, rows, scale pitch]; an expert's rows are dense."""
    mx = gate_scales is not None
    if mx and (up_scales is None or down_scales is None):
        raise ValueError("MXFP4 experts need the scales of all three matrices")
    weight, size = (_U8, 1) if mx else (_BF16, 2)
    if not (gate.dtype is weight and up.dtype is weight and down.dtype is weight
            and gate.is_contiguous() and up.is_contiguous() and down.is_contiguous()):
        _bind_types()
        for t, what in ((gate, "gate"), (up, "up"), (down, "down")):
            if (t.itemsize != 1) if mx else _is_f32(t):
                raise TypeError(f"{what} has to be {'bytes (it has scales)' if mx else 'bf16'}, not {t.dtype}")
            _expert_rows(t, what)
    # bytes between the experts of a stacked tensor (one expert's are not read)
    gs = gate.stride(0)
    if up.stride(0) != gs and E > 1:
        raise ValueError("gate and up need the same distance between experts")
    if mx:
        if not (gate_scales.dtype is _U8 and up_scales.dtype is _U8 and down_scales.dtype is _U8
                and gate_scales.is_contiguous() and up_scales.is_contiguous() and down_scales.is_contiguous()):
            for t, what in ((gate_scales, "gate_scales"), (up_scales, "up_scales"), (down_scales, "down_scales")):
                if t.itemsize != 1:
                    raise TypeError(f"{what} has to be bytes, not {t.dtype}")
                _expert_rows(t, what)
        ss = gate_scales.stride(0)
        if up_scales.stride(0) != ss and E > 1:
            raise ValueError("gate and up need the same distance between experts")
        w = _experts(1, 0, gate.data_ptr(), up.data_ptr(), down.data_ptr(), gs, down.stride(0), gate_scales.data_ptr(),
                     up_scales.data_ptr(), down_scales.data_ptr(), ss, down_scales.stride(0))
    else:
        w = _experts(0, 0, gate.data_ptr(), up.data_ptr(), down.data_ptr(), size * gs, size * down.stride(0), 0, 0, 0, 0, 0)
    try:
        usual = (x.dtype is _BF16 and out.dtype is _BF16 and logits.dtype is _F32 and x.is_contiguous()
                 and out.is_contiguous() and logits.is_contiguous())
    except AttributeError:
        usual = False
    if usual:
        px, pl, po = x.data_ptr(), logits.data_ptr(), out.data_ptr()
    else:
        px, pl, po = _values(x, 0, "x"), _values(logits, 1, "logits"), _values(out, 0, "out")
    pr = 0 if resid is None else _values(resid, 1, "resid")
    p32 = 0 if out32 is None else _values(out32, 1, "out32")
    return _check(_lib.lsk_moe_few(px, pr, pl, w, T, E, k, H, F, po, p32, _stream(stream)))


# ------------------------------------------------------------------ products whose weights differ by rows
class LoraAdapters:
    """The adapters of one projection as the library takes them, and references to their tensors."""

    def __init__(self, down, up, up2=None, scale=None):
        for t, what in ((down, "down"), (up, "up")) + (() if up2 is None else ((up2, "up2"),)):
            if _dtype_code(t) != LS_DTYPE_BF16:
                raise TypeError(f"{what} has to be bf16, not {t.dtype}")
            if t.dim() != 3:
                raise ValueError(f"{what} has to be [adapters, rows, columns]")
            _expert_rows(t, what)
        n, rank = up.shape[0], up.shape[2]
        rows = rank if up2 is None else 2 * rank
        if down.shape[0] != n or down.shape[1] != rows or (up2 is not None and up2.shape != up.shape):
            raise ValueError("the adapters' matrices do not belong together")
        if up2 is not None and n > 1 and up2.stride(0) != up.stride(0):
            raise ValueError("up and up2 need the same distance between adapters")
        self.N, self.K, self.two = up.shape[1], down.shape[2], up2 is not None
        self.keep = (down, up, up2, scale)
        if scale is not None and scale.shape != (n,):
            raise ValueError("scale has to be [adapters]")
        self.c = lsk_lora(n, rank, down.data_ptr(), up.data_ptr(), _ptr(up2), 0 if scale is None else _values(scale, 1, "scale"),
                          2 * down.stride(0), 2 * up.stride(0))
        self.ref = C.addressof(self.c)


def lsk_lora_adapters(down, up, up2=None, scale=None) -> LoraAdapters:
    """Adapters beside a projection [N, K]: down [n, rank, K] and up [n, N, rank] bf16 (the gate/up pair: down [n, 2 rank, K], the
    gate's rows first, and up2 [n, N, rank]), scale [n] float32 or None. Adapters may lie apart; the rows of each are dense."""
    return LoraAdapters(down, up, up2, scale)


def _ids(t, what: str, need: int):
    """Address of a dense int32 tensor of at least `need` values; raw addresses and None pass."""
    if getattr(t, "dtype", None) is not None:
        if t.dtype is not _INT32 and ("int32" not in str(t.dtype) or "uint" in str(t.dtype)):
            raise TypeError(f"{what} has to be int32, not {t.dtype}")
        _dense(t, what)
        if t.numel() < need:
            raise ValueError(f"{what} has {t.numel()} values, not {need}")
    return _ptr(t)


def lsk_gemm_lora_bf16(epilogue: int, A, B, adapters: LoraAdapters, ids, C_out, M: int, N: int, K: int, bias=None, resid=None,
                       b_rows: int | None = None, b2_row_off: int = 0, C32=None, stream=None) -> int:
    """lsk_gemm_bf16 with the adapter ids[t] (int32 [M], none where it is not one of the adapters') beside row t's product."""
    if adapters.N != N or adapters.K != K or adapters.two != (epilogue == LSK_EPI_SWIGLU):
        raise ValueError("these adapters are for another projection")
    try:
        usual = (A.dtype is _BF16 and B.dtype is _BF16 and C_out.dtype is _BF16 and ids.dtype is _INT32 and A.is_contiguous()
                 and B.is_contiguous() and C_out.is_contiguous() and ids.is_contiguous() and ids.numel() >= M)
    except AttributeError:
        usual = False
    if usual:
        a, b, i, c = A.data_ptr(), B.data_ptr(), ids.data_ptr(), C_out.data_ptr()
    else:
        _bind_types()
        a, b, i, c = _values(A, 0, "A"), _values(B, 0, "B"), _ids(ids, "ids", M), _values(C_out, 0, "C_out")
    rows = b_rows if b_rows is not None else B.shape[0]
    rf32 = 0 if resid is None else _is_f32(resid)
    return _check(_lib.lsk_gemm_lora_bf16(
        epilogue, a, b, rows, b2_row_off, adapters.ref, i, 0 if bias is None else _values(bias, 0, "bias"),
        0 if resid is None else _values(resid, rf32, "resid"), rf32, c, 0 if C32 is None else _values(C32, 1, "C32"), M, N, K,
        _stream(stream)))


def _packed(codes, scales, n: int, N: int, K: int, what: str):
    """Addresses of n or more stacked MXFP4 matrices, each of N rows of K values (or more rows), and the bytes between them."""
    cp, sp = (K + 127) // 128 * 64, (K + 511) // 512 * 16
    if codes.dtype is _U8 and scales.dtype is _U8 and codes.is_contiguous() and scales.is_contiguous():
        c, s = codes.stride(), scales.stride()
        if len(c) == len(s) == 3:
            cs, ss = c[0], s[0]
            if c[1] == cp and s[1] == sp and cs >= N * cp and ss >= N * sp and codes.numel() >= n * cs and scales.numel() >= n * ss:
                return codes.data_ptr(), scales.data_ptr(), cs, ss
    _bind_types()
    for t, pitch, name in ((codes, cp, what + "_codes"), (scales, sp, what + "_scales")):
        if t.itemsize != 1:
            raise TypeError(f"{name} has to be bytes, not {t.dtype}")
        _expert_rows(t, name)
        if t.shape[0] < n:
            raise ValueError(f"{name} has fewer matrices than {n} groups")
        rows = t.shape[1:]
        if (rows[1] != pitch or rows[0] < N) if len(rows) == 2 else t.numel() < t.shape[0] * N * pitch:
            raise ValueError(f"{name} of {tuple(rows)} a group are not {N} rows of {pitch} bytes")
    return codes.data_ptr(), scales.data_ptr(), codes.stride(0), scales.stride(0)


def lsk_gemm_grouped_bf16_mxfp4(epilogue: int, A, B_codes, B_scales, group_bounds, n_groups: int, C_out, M: int, N: int, K: int,
                                B2_codes=None, B2_scales=None, row_table=None, row_weight=None, gather_k: int = 0,
                                stream=None) -> int:
    """Rows sorted by group through the groups' MXFP4 matrices: B_codes [n_groups, N, code pitch] and B_scales [n_groups, N, scale pitch]
    (LSK_EPI_SWIGLU: B2 likewise), A [rows, K] bf16, group_bounds [n_groups + 1] and row_table [M] int32, row_weight [M] float32,
    C_out [M, N] bf16, float32 for LSK_EPI_SCALE_F32; all but the groups dense. gather_k > 0: row i is A's row row_table[i] // gather_k."""
    bc, bs, cs, ss = _packed(B_codes, B_scales, n_groups, N, K, "B")
    b2c = b2s = 0
    if B2_codes is not None:
        b2c, b2s, c2, s2 = _packed(B2_codes, B2_scales, n_groups, N, K, "B2")
        if (c2 != cs or s2 != ss) and n_groups > 1:
            raise ValueError("B and B2 need the same distance between groups")
    rows = A.shape
    if A.numel() != rows[0] * K and K % 8 == 0:      # (the library refuses other K)
        raise ValueError(f"A of {tuple(rows)} has no rows of {K} values")
    f32 = epilogue == LSK_EPI_SCALE_F32
    if f32 and getattr(row_weight, "dtype", None) is not None and row_weight.numel() < M:
        raise ValueError(f"row_weight has {row_weight.numel()} values, not {M}")
    try:
        usual = (A.dtype is _BF16 and C_out.dtype is (_F32 if f32 else _BF16) and group_bounds.dtype is _INT32 and A.is_contiguous()
                 and C_out.is_contiguous() and group_bounds.is_contiguous() and group_bounds.numel() > n_groups)
    except AttributeError:
        usual = False
    if usual:
        a, g, c = A.data_ptr(), group_bounds.data_ptr(), C_out.data_ptr()
    else:
        _bind_types()
        a, g, c = _values(A, 0, "A"), _ids(group_bounds, "group_bounds", n_groups + 1), _values(C_out, int(f32), "C_out")
    return _check(_lib.lsk_gemm_grouped_bf16_mxfp4(
        epilogue, a, rows[0], bc, bs, b2c, b2s, cs, ss, g, n_groups, 0 if row_table is None else _ids(row_table, "row_table", M),
        0 if row_weight is None else _values(row_weight, 1, "row_weight"), gather_k, c, M, N, K, _stream(stream)))
