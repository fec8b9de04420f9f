"""ctypes binding of the C ABI in ``include/conv3d_fp8.h``, ``include/q8.h`` and
``include/q8_attention.h`` (argument marshalling only).

Every entry point keeps its C name. Tensors are passed as raw device pointers (``data_ptr()``);
torch is only used for device memory and streams. There is no fallback of any kind: if the CUDA
library has not been built, ``load()`` raises.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

from . import build as _build

CONV3D_OK = 0
CONV3D_EINVAL = 1
CONV3D_EUNSUPPORTED = 2
CONV3D_ENOMEM = 3
CONV3D_ECUDA = 4
CONV3D_EDEVICE = 5

_lock = threading.Lock()
_lib = None


class Conv3dFp8Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {conv3d_fp8_strerror(status)} (status {status})")


class Options(ctypes.Structure):
    _fields_ = [("splits", ctypes.c_int), ("block_n", ctypes.c_int), ("max_ctas", ctypes.c_int),
                ("wait_timeout_ms", ctypes.c_int), ("debug_flags", ctypes.c_int),
                ("route", ctypes.c_int), ("cta_pair", ctypes.c_int),
                ("input_layout", ctypes.c_int), ("epilogue", ctypes.c_int),
                ("overlap", ctypes.c_int)]


class LinearOptions(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int), ("block_t", ctypes.c_int), ("splits", ctypes.c_int),
                ("max_ctas", ctypes.c_int), ("wait_timeout_ms", ctypes.c_int),
                ("debug_flags", ctypes.c_int)]


class AttnOptions(ctypes.Structure):
    _fields_ = [("wait_timeout_ms", ctypes.c_int), ("debug_flags", ctypes.c_int)]


class PlanInfo(ctypes.Structure):
    _fields_ = [("Do", ctypes.c_int), ("Ho", ctypes.c_int), ("Wo", ctypes.c_int),
                ("npq", ctypes.c_longlong), ("k_gemm", ctypes.c_int), ("block_m", ctypes.c_int),
                ("block_n", ctypes.c_int), ("m_tiles", ctypes.c_int), ("n_tiles", ctypes.c_int),
                ("k_blocks", ctypes.c_int), ("splits", ctypes.c_int),
                ("k_blocks_per_split", ctypes.c_int), ("stages", ctypes.c_int),
                ("row_chk", ctypes.c_int), ("grid", ctypes.c_int), ("sm_count", ctypes.c_int),
                ("workspace_bytes", ctypes.c_size_t), ("route", ctypes.c_int),
                ("cta_pair", ctypes.c_int), ("full_tiles", ctypes.c_int),
                ("epilogue", ctypes.c_int), ("overlap_planes", ctypes.c_int),
                ("overlap_units", ctypes.c_int)]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


def library_path() -> str:
    return _build.LIB_PATH


def load() -> ctypes.CDLL:
    """Load the in-tree CUDA library. Raises if it is missing: there is no other code path."""
    global _lib
    with _lock:
        if _lib is None:
            path = _build.LIB_PATH
            if not os.path.exists(path):
                raise RuntimeError(
                    f"CUDA library {path} is not built; run `python -m fp8_implicit_gemm_gb300.build`"
                    " (or __graft_entry__.build()) first")
            lib = ctypes.CDLL(path)
            ci, vp = ctypes.c_int, ctypes.c_void_p
            i3 = ctypes.POINTER(ctypes.c_int)
            lib.conv3d_fp8_plan.restype = ci
            lib.conv3d_fp8_plan.argtypes = [ctypes.POINTER(vp)] + [ci] * 9 + [i3, i3, ci]
            lib.conv3d_fp8_plan_ex.restype = ci
            lib.conv3d_fp8_plan_ex.argtypes = ([ctypes.POINTER(vp)] + [ci] * 9 + [i3, i3, ci]
                                               + [ctypes.POINTER(Options)])
            lib.conv3d_fp8_run.restype = ci
            lib.conv3d_fp8_run.argtypes = [vp, vp, vp, vp, vp, vp, i3, i3, vp]
            lib.conv3d_fp8_set_timing_events.restype = ci
            lib.conv3d_fp8_set_timing_events.argtypes = [vp, vp, vp]
            lib.conv3d_fp8_set_pack_timing_event.restype = ci
            lib.conv3d_fp8_set_pack_timing_event.argtypes = [vp, vp]
            lib.conv3d_fp8_set_write_counter.restype = ci
            lib.conv3d_fp8_set_write_counter.argtypes = [vp, vp]
            lib.conv3d_fp8_run_noalloc.restype = ci
            lib.conv3d_fp8_run_noalloc.argtypes = [ci] * 9 + [i3, i3, vp, vp, vp, vp, vp, vp]
            lib.conv3d_fp8_noalloc_check.restype = ci
            lib.conv3d_fp8_noalloc_check.argtypes = []
            lib.conv3d_fp8_check.restype = ci
            lib.conv3d_fp8_check.argtypes = [vp]
            lib.conv3d_fp8_get_info.restype = ci
            lib.conv3d_fp8_get_info.argtypes = [vp, ctypes.POINTER(PlanInfo)]
            lib.conv3d_fp8_describe.restype = ci
            lib.conv3d_fp8_describe.argtypes = ([ci] * 9 + [i3, i3, ci, ctypes.POINTER(Options),
                                                            ctypes.POINTER(PlanInfo)])
            lib.conv3d_bf16_plan.restype = ci
            lib.conv3d_bf16_plan.argtypes = [ctypes.POINTER(vp)] + [ci] * 9 + [i3, i3, ci]
            lib.conv3d_bf16_plan_ex.restype = ci
            lib.conv3d_bf16_plan_ex.argtypes = ([ctypes.POINTER(vp)] + [ci] * 9 + [i3, i3, ci]
                                                + [ctypes.POINTER(Options)])
            lib.conv3d_bf16_run.restype = ci
            lib.conv3d_bf16_run.argtypes = [vp, vp, vp, vp, i3, i3, vp]
            lib.conv3d_fp8_run_host.restype = ci
            lib.conv3d_fp8_run_host.argtypes = [vp, vp, vp, vp, vp, i3, i3, vp]
            lib.conv3d_bf16_run_host.restype = ci
            lib.conv3d_bf16_run_host.argtypes = [vp, vp, vp, vp, i3, i3, vp]
            lib.conv3d_bf16_describe.restype = ci
            lib.conv3d_bf16_describe.argtypes = ([ci] * 9 + [i3, i3, ci, ctypes.POINTER(Options),
                                                             ctypes.POINTER(PlanInfo)])
            lib.conv3d_fp8_quantize.restype = ci
            lib.conv3d_fp8_quantize.argtypes = [vp, ci, ctypes.c_longlong, vp, vp, vp]
            lib.conv3d_fp8_run_quantize_x.restype = ci
            lib.conv3d_fp8_run_quantize_x.argtypes = [vp, vp, ci, vp, vp, vp, i3, i3, vp, vp]
            lib.conv3d_fp8_workspace_size.restype = ctypes.c_size_t
            lib.conv3d_fp8_workspace_size.argtypes = [vp]
            lib.conv3d_fp8_out_dims.restype = ci
            lib.conv3d_fp8_out_dims.argtypes = [vp, i3, i3, i3]
            lib.conv3d_fp8_destroy.restype = None
            lib.conv3d_fp8_destroy.argtypes = [vp]
            lib.conv3d_fp8_strerror.restype = ctypes.c_char_p
            lib.conv3d_fp8_strerror.argtypes = [ci]
            cq = ctypes.c_longlong
            for name in ("rmsnorm_q8_run", "silu_mul_q8_run"):
                getattr(lib, name).restype = ci
                getattr(lib, name).argtypes = [ctypes.c_char_p]
            lib.linear_q8_plan.restype = ci
            lib.linear_q8_plan.argtypes = [ctypes.POINTER(vp), cq, cq, cq, ci, ci]
            lib.linear_q8_plan_ex.restype = ci
            lib.linear_q8_plan_ex.argtypes = ([ctypes.POINTER(vp), cq, cq, cq, ci, ci]
                                              + [ctypes.POINTER(LinearOptions)])
            lib.linear_q8_run.restype = ci
            lib.linear_q8_run.argtypes = [vp, ctypes.c_char_p]
            lib.linear_q8_check.restype = ci
            lib.linear_q8_check.argtypes = [vp]
            lib.linear_q8_workspace_size.restype = ctypes.c_size_t
            lib.linear_q8_workspace_size.argtypes = [vp]
            lib.linear_q8_destroy.restype = None
            lib.linear_q8_destroy.argtypes = [vp]
            for name in ("heads_q8_run", "cache_q8_read_run"):
                getattr(lib, name).restype = ci
                getattr(lib, name).argtypes = [ctypes.c_char_p]
            lib.attn_q8_plan.restype = ci
            lib.attn_q8_plan.argtypes = [ctypes.POINTER(vp), cq] + [ci] * 6
            lib.attn_prompt_plan.restype = ci
            lib.attn_prompt_plan.argtypes = [ctypes.POINTER(vp), ci]
            lib.attn_q8_plan_ex.restype = ci
            lib.attn_q8_plan_ex.argtypes = [ctypes.POINTER(vp), cq] + [ci] * 6 + [ctypes.POINTER(AttnOptions)]
            lib.attn_prompt_plan_ex.restype = ci
            lib.attn_prompt_plan_ex.argtypes = [ctypes.POINTER(vp), ci, ctypes.POINTER(AttnOptions)]
            for name in ("attn_q8_run", "attn_prompt_run"):
                getattr(lib, name).restype = ci
                getattr(lib, name).argtypes = [vp, ctypes.c_char_p]
            for name in ("attn_q8_check", "attn_prompt_check"):
                getattr(lib, name).restype = ci
                getattr(lib, name).argtypes = [vp]
            lib.attn_q8_workspace_size.restype = ctypes.c_size_t
            lib.attn_q8_workspace_size.argtypes = [vp]
            for name in ("attn_q8_destroy", "attn_prompt_destroy"):
                getattr(lib, name).restype = None
                getattr(lib, name).argtypes = [vp]
            _lib = lib
    return _lib


def _int3(v):
    if isinstance(v, int):
        v = (v, v, v)
    v = tuple(int(i) for i in v)
    if len(v) != 3:
        raise ValueError("expected an int or 3 ints (d, h, w)")
    return (ctypes.c_int * 3)(*v)


def _options(**kw) -> Options | None:
    if not kw:
        return None
    o = Options()
    for k, v in kw.items():
        if v is not None:
            setattr(o, k, int(v))
    return o


def _ptr(t) -> int:
    """Device address of a torch tensor (or an int address, passed through)."""
    if t is None:
        return 0
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _host_ptr(t) -> int:
    """Host address of a CPU torch tensor (or an int address, passed through)."""
    if t is None:
        return 0
    if isinstance(t, int):
        return t
    if t.is_cuda:
        raise ValueError("expected a CPU tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _raise(status: int, where: str):
    if status != CONV3D_OK:
        raise Conv3dFp8Error(status, where)


def conv3d_fp8_strerror(status: int) -> str:
    return load().conv3d_fp8_strerror(int(status)).decode()


def conv3d_fp8_plan(N, C, D, H, W, K, T, R, S, stride, pad, device=0, **options) -> int:
    """Create a plan; returns its handle. Keyword options (0 = the library's choice): splits,
    block_n, max_ctas, wait_timeout_ms, debug_flags, route, cta_pair, input_layout (1 = x is
    NDHWC), epilogue (2 = TMA-store epilogue), overlap (-1 = never pack beside the GEMM, P > 0 =
    pack P input planes before it); see conv3d_fp8_options in include/conv3d_fp8.h."""
    lib = load()
    h = ctypes.c_void_p()
    o = _options(**options)
    if o is None:
        st = lib.conv3d_fp8_plan(ctypes.byref(h), N, C, D, H, W, K, T, R, S, _int3(stride),
                                 _int3(pad), device)
    else:
        st = lib.conv3d_fp8_plan_ex(ctypes.byref(h), N, C, D, H, W, K, T, R, S, _int3(stride),
                                    _int3(pad), device, ctypes.byref(o))
    _raise(st, "conv3d_fp8_plan")
    return h.value


def conv3d_fp8_run(plan, x, w, scale_x, scale_w, y, stride, pad, stream=None) -> None:
    st = load().conv3d_fp8_run(plan, _ptr(x), _ptr(w), _ptr(scale_x), _ptr(scale_w), _ptr(y),
                               _int3(stride), _int3(pad), _stream(stream))
    _raise(st, "conv3d_fp8_run")


def conv3d_fp8_run_status(plan, x, w, scale_x, scale_w, y, stride, pad, stream=None) -> int:
    """As conv3d_fp8_run, but returns the status code instead of raising."""
    return load().conv3d_fp8_run(plan, _ptr(x), _ptr(w), _ptr(scale_x), _ptr(scale_w), _ptr(y),
                                 _int3(stride), _int3(pad), _stream(stream))


def conv3d_fp8_run_host_status(plan, x_host, w_host, scales_host, y_host, stride, pad,
                               stream=None) -> int:
    """conv3d_fp8_run_host: CPU tensors (page-locked for asynchronous copies); scales_host holds
    (scale_x, scale_w) as fp32. Returns the status code."""
    return load().conv3d_fp8_run_host(plan, _host_ptr(x_host), _host_ptr(w_host),
                                      _host_ptr(scales_host), _host_ptr(y_host), _int3(stride),
                                      _int3(pad), _stream(stream))


def conv3d_fp8_run_host(plan, x_host, w_host, scales_host, y_host, stride, pad,
                        stream=None) -> None:
    _raise(conv3d_fp8_run_host_status(plan, x_host, w_host, scales_host, y_host, stride, pad,
                                      stream), "conv3d_fp8_run_host")


def conv3d_fp8_run_noalloc_status(N, C, D, H, W, K, T, R, S, stride, pad, x, w, scale_x,
                                  scale_w, y, stream=None) -> int:
    """Allocation-free run (no plan; scratch in a fixed device array of the library, see
    include/conv3d_fp8.h). Returns the status code."""
    return load().conv3d_fp8_run_noalloc(N, C, D, H, W, K, T, R, S, _int3(stride), _int3(pad),
                                         _ptr(x), _ptr(w), _ptr(scale_x), _ptr(scale_w), _ptr(y),
                                         _stream(stream))


def conv3d_fp8_noalloc_check() -> int:
    """Synchronise the current device, then report (and clear) the status word of its latest
    allocation-free call: CONV3D_OK or CONV3D_EDEVICE."""
    return int(load().conv3d_fp8_noalloc_check())


def conv3d_fp8_run_noalloc(N, C, D, H, W, K, T, R, S, stride, pad, x, w, scale_x, scale_w, y,
                           stream=None) -> None:
    _raise(conv3d_fp8_run_noalloc_status(N, C, D, H, W, K, T, R, S, stride, pad, x, w, scale_x,
                                         scale_w, y, stream), "conv3d_fp8_run_noalloc")


def _raw_event(ev):
    if ev is None:
        return None
    if isinstance(ev, int):
        return ev
    if not ev.cuda_event:       # torch creates its event lazily, on first record
        ev.record()
    return ev.cuda_event


def conv3d_fp8_set_timing_events(plan, ev_begin, ev_end) -> None:
    """Record the given events (torch.cuda.Event or raw cudaEvent_t ints; None to clear) around
    the main kernel of every later run of the plan."""
    _raise(load().conv3d_fp8_set_timing_events(plan, _raw_event(ev_begin), _raw_event(ev_end)),
           "conv3d_fp8_set_timing_events")


def conv3d_fp8_set_write_counter_status(plan, counts) -> int:
    """Count the stores to each output element into `counts` (a zeroed uint32/int32 device
    tensor of N*K*Do*Ho*Wo elements; None stops); only a library built with C3D_COUNT_WRITES
    counts, the product build returns CONV3D_EUNSUPPORTED."""
    return load().conv3d_fp8_set_write_counter(plan, _ptr(counts) if counts is not None else None)


def conv3d_fp8_set_pack_timing_event(plan, ev_pack) -> None:
    """Record the given event (None to clear) right before the pack kernel of every later run
    of the plan; with the begin event of conv3d_fp8_set_timing_events it brackets the pack."""
    _raise(load().conv3d_fp8_set_pack_timing_event(plan, _raw_event(ev_pack)),
           "conv3d_fp8_set_pack_timing_event")


def conv3d_fp8_check(plan) -> int:
    """Synchronise and return (and clear) the plan's device status: CONV3D_OK or CONV3D_EDEVICE."""
    return load().conv3d_fp8_check(plan)


def conv3d_fp8_get_info(plan) -> dict:
    info = PlanInfo()
    _raise(load().conv3d_fp8_get_info(plan, ctypes.byref(info)), "conv3d_fp8_get_info")
    return info.as_dict()


def conv3d_fp8_describe(N, C, D, H, W, K, T, R, S, stride, pad, sm_count, **options) -> dict:
    """Host-only planning decision (no device access)."""
    info = PlanInfo()
    o = _options(**options)
    st = load().conv3d_fp8_describe(N, C, D, H, W, K, T, R, S, _int3(stride), _int3(pad),
                                    sm_count, ctypes.byref(o) if o is not None else None,
                                    ctypes.byref(info))
    _raise(st, "conv3d_fp8_describe")
    return info.as_dict()


def conv3d_fp8_describe_status(N, C, D, H, W, K, T, R, S, stride, pad, sm_count, **options) -> int:
    info = PlanInfo()
    o = _options(**options)
    return load().conv3d_fp8_describe(N, C, D, H, W, K, T, R, S, _int3(stride), _int3(pad),
                                      sm_count, ctypes.byref(o) if o is not None else None,
                                      ctypes.byref(info))


def conv3d_fp8_workspace_size(plan) -> int:
    return int(load().conv3d_fp8_workspace_size(plan))


def conv3d_fp8_out_dims(plan) -> tuple[int, int, int]:
    d, h, w = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    _raise(load().conv3d_fp8_out_dims(plan, ctypes.byref(d), ctypes.byref(h), ctypes.byref(w)),
           "conv3d_fp8_out_dims")
    return d.value, h.value, w.value


def conv3d_fp8_destroy(plan) -> None:
    if plan:
        load().conv3d_fp8_destroy(plan)


# ------------------------------------------------------------------------- BF16-input twin
def conv3d_bf16_plan(N, C, D, H, W, K, T, R, S, stride, pad, device=0, **options) -> int:
    """Create a plan of the BF16-input twin (same options as conv3d_fp8_plan)."""
    lib = load()
    h = ctypes.c_void_p()
    o = _options(**options)
    if o is None:
        st = lib.conv3d_bf16_plan(ctypes.byref(h), N, C, D, H, W, K, T, R, S, _int3(stride),
                                  _int3(pad), device)
    else:
        st = lib.conv3d_bf16_plan_ex(ctypes.byref(h), N, C, D, H, W, K, T, R, S, _int3(stride),
                                     _int3(pad), device, ctypes.byref(o))
    _raise(st, "conv3d_bf16_plan")
    return h.value


def conv3d_bf16_run_status(plan, x, w, y, stride, pad, stream=None) -> int:
    return load().conv3d_bf16_run(plan, _ptr(x), _ptr(w), _ptr(y), _int3(stride), _int3(pad),
                                  _stream(stream))


def conv3d_bf16_run(plan, x, w, y, stride, pad, stream=None) -> None:
    _raise(conv3d_bf16_run_status(plan, x, w, y, stride, pad, stream), "conv3d_bf16_run")


def conv3d_bf16_run_host_status(plan, x_host, w_host, y_host, stride, pad, stream=None) -> int:
    return load().conv3d_bf16_run_host(plan, _host_ptr(x_host), _host_ptr(w_host),
                                       _host_ptr(y_host), _int3(stride), _int3(pad),
                                       _stream(stream))


def conv3d_bf16_run_host(plan, x_host, w_host, y_host, stride, pad, stream=None) -> None:
    _raise(conv3d_bf16_run_host_status(plan, x_host, w_host, y_host, stride, pad, stream),
           "conv3d_bf16_run_host")


def conv3d_bf16_describe_status(N, C, D, H, W, K, T, R, S, stride, pad, sm_count,
                                **options) -> int:
    info = PlanInfo()
    o = _options(**options)
    return load().conv3d_bf16_describe(N, C, D, H, W, K, T, R, S, _int3(stride), _int3(pad),
                                       sm_count, ctypes.byref(o) if o is not None else None,
                                       ctypes.byref(info))


def conv3d_bf16_describe(N, C, D, H, W, K, T, R, S, stride, pad, sm_count, **options) -> dict:
    """Host-only planning decision of the BF16-input twin (no device access)."""
    info = PlanInfo()
    o = _options(**options)
    st = load().conv3d_bf16_describe(N, C, D, H, W, K, T, R, S, _int3(stride), _int3(pad),
                                     sm_count, ctypes.byref(o) if o is not None else None,
                                     ctypes.byref(info))
    _raise(st, "conv3d_bf16_describe")
    return info.as_dict()


# ------------------------------------------------------------------------------- quantiser
CONV3D_SRC_F32 = 1
CONV3D_SRC_BF16 = 2


def _src_type(t) -> int:
    import torch
    if t.dtype == torch.float32:
        return CONV3D_SRC_F32
    if t.dtype == torch.bfloat16:
        return CONV3D_SRC_BF16
    raise ValueError(f"the quantiser takes fp32 or bfloat16 values, not {t.dtype}")


def conv3d_fp8_quantize_status(src, dst, scale_out, stream=None) -> int:
    """Quantise a CUDA fp32/bfloat16 tensor into uint8 e4m3 codes (dst) and a device scale."""
    return load().conv3d_fp8_quantize(_ptr(src), _src_type(src), src.numel(), _ptr(dst),
                                      _ptr(scale_out), _stream(stream))


def conv3d_fp8_quantize(src, dst, scale_out, stream=None) -> None:
    _raise(conv3d_fp8_quantize_status(src, dst, scale_out, stream), "conv3d_fp8_quantize")


def conv3d_fp8_run_quantize_x_status(plan, x_src, w, scale_w, y, stride, pad, scale_x_out=None,
                                     stream=None) -> int:
    return load().conv3d_fp8_run_quantize_x(plan, _ptr(x_src), _src_type(x_src), _ptr(w),
                                            _ptr(scale_w), _ptr(y), _int3(stride), _int3(pad),
                                            _ptr(scale_x_out), _stream(stream))


def conv3d_fp8_run_quantize_x(plan, x_src, w, scale_w, y, stride, pad, scale_x_out=None,
                              stream=None) -> None:
    _raise(conv3d_fp8_run_quantize_x_status(plan, x_src, w, scale_w, y, stride, pad, scale_x_out,
                                            stream), "conv3d_fp8_run_quantize_x")


# --------------------------------------------------- 8-bit codes with scales (include/q8.h)
Q8_F32, Q8_BF16, Q8_F16 = 1, 2, 3
Q8_INT8, Q8_E4M3 = 1, 2

# The argument structs of include/q8.h, packed as C lays them out on a 64-bit host: one bytes object
# crosses the boundary. These calls run once or more a layer and token, so what they check of a tensor
# is asked for once and compared in as few steps as possible.
_RMSNORM_ARGS = struct.Struct("@6P4q2qP4ifi")
_SILU_MUL_ARGS = struct.Struct("@4P3q2qP4i")
_LINEAR_ARGS = struct.Struct("@6P6qP4i")

_value_types = {}
_code_types = {}
# Set by the first call: the library, some of torch's types and its current stream's handle. These calls cost
# the host more than the GPU where there are few tokens, so nothing is looked up twice in them.
_q8 = _f32 = _i32 = _i64 = _raw_stream = None


def _q8_setup():
    global _q8, _f32, _i32, _i64, _raw_stream
    import torch
    lib = load()
    _f32, _raw_stream = torch.float32, torch._C._cuda_getCurrentRawStream
    _i32, _i64 = torch.int32, torch.int64
    _value_types.update({torch.float32: Q8_F32, torch.bfloat16: Q8_BF16, torch.float16: Q8_F16})
    _code_types.update({torch.int8: Q8_INT8, torch.uint8: Q8_E4M3, torch.float8_e4m3fn: Q8_E4M3})
    _q8 = lib
    return lib


def q8_code_type(dtype) -> int:
    """Q8_INT8 for torch.int8, Q8_E4M3 for torch.float8_e4m3fn or torch.uint8 (e4m3 bytes)."""
    t = _code_types.get(dtype)
    if t is None and not _code_types:
        _q8_setup()
        t = _code_types.get(dtype)
    if t is None:
        raise ValueError(f"codes are int8, float8_e4m3fn or uint8 (e4m3 bytes), not {dtype}")
    return t


def _q8_value_type(t, name) -> int:
    v = _value_types.get(t.dtype)
    if v is None:
        raise ValueError(f"{name} holds fp32, bfloat16 or float16 values, not {t.dtype}")
    return v


def _q8_pitch(t, name, shape, device) -> int:
    """Pitch of a matrix of this shape and device whose rows are contiguous."""
    if t.shape != shape:
        raise ValueError(f"{name}: expected the shape {tuple(shape)}, got {tuple(t.shape)}")
    pitch, step = t.stride()
    if step != 1 and t.shape[1] > 1:
        raise ValueError(f"{name}: expected contiguous rows")
    if t.get_device() != device:
        raise ValueError(f"{name}: expected a tensor on CUDA device {device}")
    return pitch


def _q8_vector(t, name, size, device, dtype=None) -> int:
    """Address of a contiguous vector of this size and device."""
    if t.shape != (size,) or not t.is_contiguous():
        raise ValueError(f"{name}: expected {size} contiguous elements")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name}: expected a tensor on CUDA device {device}")
    return t.data_ptr()


def _q8_head(t, name):
    """Shape, device and pitch of a call's first matrix."""
    shape, device = t.shape, t.get_device()
    if len(shape) != 2:
        raise ValueError(f"{name}: expected a matrix")
    if device < 0:
        raise ValueError(f"{name}: expected a CUDA tensor")
    pitch, step = t.stride()
    if step != 1 and shape[1] > 1:
        raise ValueError(f"{name}: expected contiguous rows")
    return shape, device, pitch


def _q8_stream(stream, device) -> int:
    if stream is None:
        return _raw_stream(device)
    return stream if isinstance(stream, int) else stream.cuda_stream


def rmsnorm_q8_run(x, weight, q, scale, eps, residual=None, residual_out=None,
                   stream=None) -> None:
    """h = x + residual; residual_out = h; q, scale = the codes of h / rms(h) * weight, a scale a
    row. Matrices [rows, cols] with contiguous rows (any pitch); the codes' type is q's."""
    lib = _q8 or _q8_setup()
    shape, device, x_pitch = _q8_head(x, "x")
    rows, cols = shape
    value_type = _q8_value_type(x, "x")
    r_ptr = out_ptr = r_pitch = out_pitch = 0
    if residual is not None:
        if residual.dtype != x.dtype:
            raise ValueError(f"residual: expected {x.dtype}, got {residual.dtype}")
        r_pitch, r_ptr = _q8_pitch(residual, "residual", shape, device), residual.data_ptr()
    if residual_out is residual:
        out_pitch, out_ptr = r_pitch, r_ptr
    elif residual_out is not None:
        if residual_out.dtype != x.dtype:
            raise ValueError(f"residual_out: expected {x.dtype}, got {residual_out.dtype}")
        out_pitch = _q8_pitch(residual_out, "residual_out", shape, device)
        out_ptr = residual_out.data_ptr()
    status = lib.rmsnorm_q8_run(_RMSNORM_ARGS.pack(
        x.data_ptr(), r_ptr, _q8_vector(weight, "weight", cols, device), out_ptr, q.data_ptr(),
        _q8_vector(scale, "scale", rows, device, _f32), x_pitch, r_pitch, out_pitch,
        _q8_pitch(q, "q", shape, device), rows, cols, _q8_stream(stream, device),
        value_type, _q8_value_type(weight, "weight"), q8_code_type(q.dtype), device, eps, 0))
    if status:
        _raise(status, "rmsnorm_q8_run")


def silu_mul_q8_run(gate, up, q, scale, stream=None) -> None:
    """q, scale = the codes of silu(gate) * up, a scale a row. Matrices [rows, cols] with contiguous
    rows (any pitch; gate and up may be two halves of one matrix); the codes' type is q's."""
    lib = _q8 or _q8_setup()
    shape, device, gate_pitch = _q8_head(gate, "gate")
    rows, cols = shape
    value_type = _q8_value_type(gate, "gate")
    if up.dtype != gate.dtype:
        raise ValueError(f"up: expected {gate.dtype}, got {up.dtype}")
    status = lib.silu_mul_q8_run(_SILU_MUL_ARGS.pack(
        gate.data_ptr(), up.data_ptr(), q.data_ptr(),
        _q8_vector(scale, "scale", rows, device, _f32), gate_pitch,
        _q8_pitch(up, "up", shape, device), _q8_pitch(q, "q", shape, device), rows, cols,
        _q8_stream(stream, device), value_type, q8_code_type(q.dtype), device, 0))
    if status:
        _raise(status, "silu_mul_q8_run")


def linear_q8_plan(max_rows, N, K, code_type, device=0, **options) -> int:
    """Create a plan for products of up to max_rows tokens by an [N, K] weight (code_type: Q8_INT8
    or Q8_E4M3); returns its handle. Keyword options (0 = the library's choice): kernel, block_t,
    splits, max_ctas, wait_timeout_ms, debug_flags; see linear_q8_options in include/q8.h."""
    lib = load()
    h = ctypes.c_void_p()
    if not options:
        st = lib.linear_q8_plan(ctypes.byref(h), max_rows, N, K, code_type, device)
    else:
        o = LinearOptions(**{k: int(v) for k, v in options.items()})
        st = lib.linear_q8_plan_ex(ctypes.byref(h), max_rows, N, K, code_type, device,
                                   ctypes.byref(o))
    _raise(st, "linear_q8_plan")
    return h.value


def linear_q8_weights(w, scale_w, bias=None) -> tuple:
    """What linear_q8_run_weights needs of a layer's weights w [N, K], scale_w [N] and bias [N],
    checked once. The caller keeps the tensors alive and where they are."""
    _q8 or _q8_setup()
    shape, device, w_pitch = _q8_head(w, "w")
    N, K = shape
    b_ptr = b_type = 0
    if bias is not None:
        b_ptr = _q8_vector(bias, "bias", N, device)
        b_type = _q8_value_type(bias, "bias")
    return (w.data_ptr(), w_pitch, _q8_vector(scale_w, "scale_w", N, device, _f32), b_ptr, b_type,
            N, K, q8_code_type(w.dtype), device)


def linear_q8_run_weights(plan, x, scale_x, weights, y, stream=None) -> None:
    """linear_q8_run on weights checked before: for few tokens the checks of all tensors take the
    host as long as the rest of the call."""
    w_ptr, w_pitch, scale_w_ptr, b_ptr, b_type, N, K, code_type, device = weights
    x_shape, x_device, x_pitch = _q8_head(x, "x")
    rows = x_shape[0]
    if x_shape[1] != K or x_device != device:
        raise ValueError(f"x: expected {K} columns on CUDA device {device}, got {x_shape[1]} on "
                         f"{x_device}")
    if q8_code_type(x.dtype) != code_type:
        raise ValueError(f"x and w hold codes of one type, not {x.dtype} and another")
    status = _q8.linear_q8_run(plan, _LINEAR_ARGS.pack(
        x.data_ptr(), _q8_vector(scale_x, "scale_x", rows, device, _f32), w_ptr, scale_w_ptr, b_ptr,
        y.data_ptr(), x_pitch, w_pitch, _q8_pitch(y, "y", (rows, N), device), rows, N, K,
        _q8_stream(stream, device), _q8_value_type(y, "y"), b_type, code_type, 0))
    if status:
        _raise(status, "linear_q8_run")


def linear_q8_run(plan, x, scale_x, w, scale_w, y, bias=None, stream=None) -> None:
    """y[m, n] = scale_x[m] * scale_w[n] * sum_k x[m, k] * w[n, k] + bias[n]. x [rows, K] and
    w [N, K] are codes of one type with row pitches that are multiples of 16, y is [rows, N]."""
    linear_q8_run_weights(plan, x, scale_x, linear_q8_weights(w, scale_w, bias), y, stream)


def linear_q8_check(plan) -> int:
    """Synchronise and return (and clear) the plan's device status: CONV3D_OK or CONV3D_EDEVICE."""
    return load().linear_q8_check(plan)


def linear_q8_workspace_size(plan) -> int:
    return int(load().linear_q8_workspace_size(plan))


def linear_q8_destroy(plan) -> None:
    if plan:
        load().linear_q8_destroy(plan)


# -------------------------------------- heads, caches and attention (include/q8_attention.h)
Q8_INT4 = 3

_CACHE = struct.Struct("@4Pq4i")
_HEADS_ARGS = struct.Struct("@12P12qP9if")
_CACHE_READ_ARGS = struct.Struct("@4P5qP2i")
_ATTN_ARGS = struct.Struct("@5P7qP3if")
_ATTN_PROMPT_ARGS = struct.Struct("@6P11qP5if")


def cache_q8(k_codes, k_scale, v_codes, v_scale) -> tuple:
    """What the calls on a cache need of its tensors, checked once: codes [pages, kv_heads, page_size,
    head_dim] (int8, float8_e4m3fn, or uint8 e4m3 bytes) with scales [pages, kv_heads, page_size], or 4-bit codes
    [.., head_dim / 2] uint8 with scales [pages, kv_heads, page_size, 2]. The caller keeps the tensors alive
    and where they are, and the tuple as long as it is used."""
    _q8 or _q8_setup()
    shape, device = k_codes.shape, k_codes.get_device()
    if len(shape) != 4:
        raise ValueError("k_codes: expected [pages, kv_heads, page_size, head_dim]")
    if device < 0:
        raise ValueError("k_codes: expected a CUDA tensor")
    pages, kv_heads, page_size, width = shape
    four = k_scale.dim() == 4
    if four:
        import torch
        if k_codes.dtype != torch.uint8:
            raise ValueError(f"k_codes: 4-bit codes lie in uint8 bytes, not {k_codes.dtype}")
        code_type, head_dim = Q8_INT4, 2 * width
    else:
        code_type, head_dim = q8_code_type(k_codes.dtype), width
    for t, name, want, dtype in ((k_codes, "k_codes", shape, k_codes.dtype),
                                 (v_codes, "v_codes", shape, k_codes.dtype),
                                 (k_scale, "k_scale", shape[:3] + (2,) * four, _f32),
                                 (v_scale, "v_scale", shape[:3] + (2,) * four, _f32)):
        if t.shape != want or t.dtype != dtype or not t.is_contiguous() or t.get_device() != device:
            raise ValueError(f"{name}: expected {tuple(want)}, contiguous, {dtype}, on CUDA device {device}")
        if t.data_ptr() % 16:
            raise ValueError(f"{name}: expected a tensor on 16 bytes")
    if (page_size % 16 or head_dim not in (64, 128, 256) or not 0 < pages * page_size < 1 << 31
            or not 0 < kv_heads < 1 << 15):
        raise ValueError(f"k_codes: expected pages of a multiple of 16 tokens, fewer than 2^31 in all, and heads of 64, 128 or "
                         f"256, got {pages} pages of {page_size}, {kv_heads} heads of {head_dim}")
    packed = ctypes.create_string_buffer(_CACHE.pack(
        k_codes.data_ptr(), v_codes.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), pages, page_size,
        kv_heads, head_dim, code_type), _CACHE.size)
    return ctypes.addressof(packed), kv_heads, head_dim, code_type, device, packed


def _heads(t, name, shape, dtype, device):
    """Address, pitch and head pitch of a matrix of heads [tokens, heads, head_dim]."""
    if t.dtype != dtype or t.get_device() != device or t.shape != shape:
        raise ValueError(f"{name}: expected {tuple(shape)}, {dtype}, on CUDA device {device}, got "
                         f"{tuple(t.shape)}, {t.dtype}, device {t.get_device()}")
    pitch, head_pitch, step = t.stride()
    if step != 1 and shape[2] > 1:
        raise ValueError(f"{name}: expected contiguous heads")
    return t.data_ptr(), pitch, head_pitch


_NO_HEADS = (0, 0, 0)


def heads_q8_run(q=None, q_out=None, k=None, k_out=None, v=None, q_weight=None, k_weight=None,
                 eps=1e-6, rotary=None, positions=None, cache=None, slots=None, stream=None) -> None:
    """Query and key heads [tokens, heads, head_dim] normed (with a weight [head_dim]), rotated (with a
    q8.Rotary and positions [tokens] or [axes, tokens], int64) and written to q_out and k_out; with a
    cache (q8.CacheQ8, or cache_q8's tuple) k's codes and v's go to the tokens' slots (int64). See
    heads_q8_run in include/q8_attention.h."""
    lib = _q8 or _q8_setup()
    if q is not None and k is not None and q.shape[1] == 0:  # a product that left keys and values only
        q = q_out = None
    lead = q if q is not None else k
    if lead is None:
        raise ValueError("expected q or k")
    if len(lead.shape) != 3:
        raise ValueError("expected heads [tokens, heads, head_dim]")
    tokens, _, dim = lead.shape
    dtype, device = lead.dtype, lead.get_device()
    if device < 0:
        raise ValueError("expected CUDA tensors")
    value_type = _q8_value_type(lead, "q" if q is not None else "k")
    qs = qo = ks = ko = vs = _NO_HEADS
    q_heads = kv_heads = weight_type = qw = kw = 0
    if q is not None:
        shape = q.shape
        q_heads = shape[1]
        qs = _heads(q, "q", shape, dtype, device)
        if q_out is None:
            raise ValueError("q_out: expected with q")
        qo = qs if q_out is q else _heads(q_out, "q_out", shape, dtype, device)
    elif q_out is not None or q_weight is not None:
        raise ValueError("q: expected with q_out or q_weight")
    if k is not None:
        if len(k.shape) != 3:
            raise ValueError("k: expected [tokens, heads, head_dim]")
        shape = (tokens, k.shape[1], dim)
        kv_heads = k.shape[1]
        ks = _heads(k, "k", shape, dtype, device)
        if k_out is not None:
            ko = ks if k_out is k else _heads(k_out, "k_out", shape, dtype, device)
        if v is not None:
            vs = _heads(v, "v", shape, dtype, device)
    elif k_out is not None or k_weight is not None or v is not None:
        raise ValueError("k: expected with k_out, k_weight or v")
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None:
            t = _q8_value_type(w, name)
            if weight_type and t != weight_type:
                raise ValueError("q_weight and k_weight: expected one type")
            weight_type = t
    if q_weight is not None:
        qw = _q8_vector(q_weight, "q_weight", dim, device)
    if k_weight is not None:
        kw = _q8_vector(k_weight, "k_weight", dim, device)
    turns = axis = rot = pos = pos_pitch = adjacent = 0
    axes = 1
    if rotary is not None:
        turns, axis, rot, axes, adjacent, rotary_device = rotary.table
        if rotary_device != device:
            raise ValueError(f"rotary: expected one on CUDA device {device}")
        if positions is None:
            raise ValueError("positions: expected with a rotary")
        shape = positions.shape
        if len(shape) == 1 and axes == 1:
            pos = _q8_vector(positions, "positions", tokens, device, _i64)
        else:
            if (shape != (axes, tokens) or positions.dtype != _i64 or positions.get_device() != device
                    or (tokens > 1 and positions.stride(1) != 1)):
                raise ValueError(f"positions: expected ({axes}, {tokens}), int64, on CUDA device {device}")
            pos, pos_pitch = positions.data_ptr(), positions.stride(0)
    elif positions is not None:
        raise ValueError("rotary: expected with positions")
    cache_ptr = slot_ptr = 0
    if cache is not None:
        cache = cache if cache.__class__ is tuple else cache.parts
        if slots is None or v is None:
            raise ValueError("v and slots: expected with a cache")
        if cache[4] != device:
            raise ValueError(f"cache: expected one on CUDA device {device}")
        cache_ptr, slot_ptr = cache[0], _q8_vector(slots, "slots", tokens, device, _i64)
    elif slots is not None or v is not None:
        raise ValueError("cache: expected with v or slots")
    if tokens == 0:
        return
    status = lib.heads_q8_run(_HEADS_ARGS.pack(
        qs[0], qo[0], ks[0], ko[0], vs[0], qw, kw, turns, axis, pos, slot_ptr, cache_ptr, qs[1], qs[2], qo[1],
        qo[2], ks[1], ks[2], ko[1], ko[2], vs[1], vs[2], pos_pitch, tokens, _q8_stream(stream, device), q_heads,
        kv_heads, dim, rot, axes, adjacent, value_type, weight_type, device, eps))
    if status:
        _raise(status, "heads_q8_run")


def cache_q8_read_run(cache, slots, k, v, stream=None) -> None:
    """k and v [tokens, kv_heads, head_dim] = the cache's values at the slots [tokens] (int64); rows of
    slots outside the cache stay as they were."""
    lib = _q8 or _q8_setup()
    cache_ptr, kv_heads, dim, _, device, _ = cache if cache.__class__ is tuple else cache.parts
    tokens = slots.shape[0]
    shape = (tokens, kv_heads, dim)
    ks, vs = _heads(k, "k", shape, k.dtype, device), _heads(v, "v", shape, k.dtype, device)
    status = lib.cache_q8_read_run(_CACHE_READ_ARGS.pack(
        cache_ptr, _q8_vector(slots, "slots", tokens, device, _i64), ks[0], vs[0], ks[1], ks[2], vs[1], vs[2], tokens,
        _q8_stream(stream, device), _q8_value_type(k, "k"), device))
    if status:
        _raise(status, "cache_q8_read_run")


# The devices of the attention plans: their runs get nothing else that says where the tensors lie.
_attn_devices = {}


def attn_q8_plan(max_seqs, max_tokens, q_heads, kv_heads, head_dim, code_type, device=0, **options) -> int:
    """Create a plan for attention of up to max_tokens newest tokens of each of up to max_seqs sequences
    over a cache (code_type: Q8_INT8, Q8_E4M3 or Q8_INT4); returns its handle. Keyword options:
    wait_timeout_ms, debug_flags; see attn_options in include/q8_attention.h."""
    h = ctypes.c_void_p()
    o = AttnOptions(**{k: int(v) for k, v in options.items()})
    _raise(load().attn_q8_plan_ex(ctypes.byref(h), max_seqs, max_tokens, q_heads, kv_heads, head_dim, code_type,
                                  device, ctypes.byref(o)), "attn_q8_plan")
    _attn_devices[h.value] = device
    return h.value


def _q8_index(t, name, device):
    """Refuses what is not int32 on the device with contiguous rows."""
    if t.dtype != _i32 or t.get_device() != device or (t.shape[-1] > 1 and t.stride(-1) != 1):
        raise ValueError(f"{name}: expected contiguous int32 on CUDA device {device}")


def attn_q8_run(plan, q, cache, table, lengths, o, scale, tokens=1, stream=None) -> None:
    """o = attention of q [seqs * tokens, q_heads, head_dim] over the cache: sequence b's place s lies in page
    table[b, s // page_size] (int32 [seqs, width]), lengths [seqs] (int32) count the newest tokens too. See
    attn_q8_run in include/q8_attention.h."""
    lib = _q8 or _q8_setup()
    cache_ptr, _, dim, _, device, _ = cache if cache.__class__ is tuple else cache.parts
    shape = q.shape
    if _attn_devices.get(plan, device) != device:
        raise ValueError(f"cache: expected one on the plan's CUDA device {_attn_devices[plan]}, got one on {device}")
    if len(shape) != 3 or shape[2] != dim or len(table.shape) != 2:
        raise ValueError(f"expected q [seqs * tokens, q_heads, {dim}] and table [seqs, width]")
    seqs, width = table.shape
    if shape[0] != seqs * tokens or lengths.shape != (seqs,):
        raise ValueError(f"expected {seqs} lengths and {seqs * tokens} rows of q, got "
                         f"{tuple(lengths.shape)} and {shape[0]}")
    dtype = q.dtype
    qs = _heads(q, "q", shape, dtype, device)
    os_ = qs if o is q else _heads(o, "o", shape, dtype, device)
    _q8_index(table, "table", device)
    _q8_index(lengths, "lengths", device)
    status = lib.attn_q8_run(plan, _ATTN_ARGS.pack(
        cache_ptr, qs[0], os_[0], table.data_ptr(), lengths.data_ptr(), qs[1], qs[2], os_[1], os_[2], seqs, width,
        table.stride(0), _q8_stream(stream, device), tokens, shape[1], _q8_value_type(q, "q"), scale))
    if status:
        _raise(status, "attn_q8_run")


def attn_q8_check(plan) -> int:
    """Synchronise and return (and clear) the plan's device status: CONV3D_OK or CONV3D_EDEVICE."""
    return load().attn_q8_check(plan)


def attn_q8_workspace_size(plan) -> int:
    return int(load().attn_q8_workspace_size(plan))


def attn_q8_destroy(plan) -> None:
    if plan:
        _attn_devices.pop(plan, None)
        load().attn_q8_destroy(plan)


def attn_prompt_plan(device=0, **options) -> int:
    """Create a plan for attention over prompts; returns its handle. Options as attn_q8_plan's."""
    h = ctypes.c_void_p()
    o = AttnOptions(**{k: int(v) for k, v in options.items()})
    _raise(load().attn_prompt_plan_ex(ctypes.byref(h), device, ctypes.byref(o)), "attn_prompt_plan")
    _attn_devices[h.value] = device
    return h.value


def attn_prompt_run(plan, q, k, v, starts, o, scale, causal=True, key_starts=None, stream=None) -> None:
    """o = attention of packed sequences: q [q_rows, q_heads, head_dim], k and v [k_rows, kv_heads,
    head_dim], starts (and key_starts) [seqs + 1] int32. See attn_prompt_run in include/q8_attention.h."""
    lib = _q8 or _q8_setup()
    device, dtype, shape = q.get_device(), q.dtype, q.shape
    if len(shape) != 3 or len(k.shape) != 3:
        raise ValueError("expected heads [rows, heads, head_dim]")
    if device < 0:
        raise ValueError("q: expected a CUDA tensor")
    if _attn_devices.get(plan, device) != device:
        raise ValueError(f"q: expected a tensor on the plan's CUDA device {_attn_devices[plan]}, got one on {device}")
    rows, heads, dim = shape
    k_rows, kv_heads, _ = k.shape
    k_shape = (k_rows, kv_heads, dim)
    qs, os_ = _heads(q, "q", shape, dtype, device), _heads(o, "o", shape, dtype, device)
    ks, vs = _heads(k, "k", k_shape, dtype, device), _heads(v, "v", k_shape, dtype, device)
    if len(starts.shape) != 1 or starts.shape[0] < 1:
        raise ValueError("starts: expected [seqs + 1]")
    _q8_index(starts, "starts", device)
    ks_ptr = 0
    if key_starts is not None:
        if key_starts.shape != starts.shape:
            raise ValueError("key_starts: expected the shape of starts")
        _q8_index(key_starts, "key_starts", device)
        ks_ptr = key_starts.data_ptr()
    elif k_rows != rows:
        raise ValueError(f"key_starts: expected with {k_rows} rows of k and {rows} of q")
    status = lib.attn_prompt_run(plan, _ATTN_PROMPT_ARGS.pack(
        qs[0], ks[0], vs[0], os_[0], starts.data_ptr(), ks_ptr, qs[1], qs[2], ks[1], ks[2], vs[1], vs[2], os_[1],
        os_[2], rows, k_rows, starts.shape[0] - 1, _q8_stream(stream, device), heads, kv_heads, dim,
        _q8_value_type(q, "q"), 1 if causal else 0, scale))
    if status:
        _raise(status, "attn_prompt_run")


def attn_prompt_check(plan) -> int:
    """Synchronise and return (and clear) the plan's device status: CONV3D_OK or CONV3D_EDEVICE."""
    return load().attn_prompt_check(plan)


def attn_prompt_destroy(plan) -> None:
    if plan:
        _attn_devices.pop(plan, None)
        load().attn_prompt_destroy(plan)
