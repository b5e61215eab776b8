"""Python binding of libbsmm (the block-scaled matmul for MI355X).

Argument marshalling only: every step of the computation runs in the HIP
kernels of ``libbsmm.so``.  The functions take PyTorch tensors (PyTorch is
used for device memory and streams), check shapes the way ``_scaled_mm``
states its scaling rules (ValueError), and pass raw pointers, strides and the
current HIP stream to the C ABI in ``include/bsmm.h``.  There is no fallback:
if the library is not built, every call raises.
"""

from __future__ import annotations

import ctypes
import os
import threading
from typing import NamedTuple

__all__ = [
    "load", "lib_path", "BsmmError",
    "bsmm_int8_rowwise", "bsmm_fp8_blockwise", "bsmm_fp8_blockwise_scratch",
    "bsmm_fp8_mx_bmm", "bsmm_fp8_scaled_mm",
    "bsmm_fp8_mx32_mm", "OP_FP8_MX32_MM", "bsmm_fp8_groupwise", "OP_FP8_GROUPWISE",
    "bsmm_quant_int8_rowwise", "bsmm_quant_fp8_blockwise", "bsmm_quant_fp8_mx",
    "bsmm_quant_fp8_columns", "bsmm_quant_fp8_weight", "bsmm_quant_fp8_blockwise_columns",
    "bsmm_quant_w4", "bsmm_w4_mm", "bsmm_w4_expert_mm",
    "bsmm_expert_mm", "bsmm_expert_wgrad",
    "bsmm_quant_int8_mx", "bsmm_swiglu", "bsmm_swiglu_backward",
    "bsmm_expert_mm_workspace_bytes", "bsmm_expert_wgrad_workspace_bytes",
    "bsmm_expert_mm_plan_name", "bsmm_expert_wgrad_plan_name",
    "bsmm_route_topk", "bsmm_route_topk_backward", "Route",
    "bsmm_w4_workspace_bytes", "bsmm_w4_plan_name", "bsmm_route_workspace_bytes",
    "bsmm_workspace_bytes", "bsmm_query_plan", "bsmm_set_override", "bsmm_set_override_tail", "bsmm_set_streamk_grid", "bsmm_mfma_probe",
    "bsmm_variant_names", "bsmm_version", "bsmm_timing_enable", "bsmm_timing_read",
    "I32", "F32", "BF16", "E4M3", "OP_INT8_ROWWISE", "OP_FP8_BLOCKWISE", "OP_FP8_MX_BMM",
    "OP_FP8_SCALED_MM",
    "STATUS",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
# BSMM_LIB_PATH: another build of the same library (the sanitized host
# build) in place of the in-tree one
lib_path = os.environ.get("BSMM_LIB_PATH") or os.path.join(_PKG, "libbsmm.so")

I32, F32, BF16, E4M3 = 0, 1, 2, 3
OP_INT8_ROWWISE, OP_FP8_BLOCKWISE, OP_FP8_MX_BMM, OP_FP8_SCALED_MM, OP_FP8_MX32_MM = 0, 1, 2, 3, 4
OP_FP8_GROUPWISE = 5
STATUS = {0: "BSMM_OK", 1: "BSMM_ERR_NULL", 2: "BSMM_ERR_SHAPE",
          3: "BSMM_ERR_SCALE_SHAPE", 4: "BSMM_ERR_LAYOUT", 5: "BSMM_ERR_ALIGN",
          6: "BSMM_ERR_DTYPE", 7: "BSMM_ERR_UNSUPPORTED", 8: "BSMM_ERR_HIP",
          9: "BSMM_ERR_ARG"}

_lib = None


class BsmmError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


class PlanInfo(ctypes.Structure):
    _fields_ = [("variant", ctypes.c_char * 48), ("tile_m", ctypes.c_int32),
                ("tile_n", ctypes.c_int32), ("split_k", ctypes.c_int32),
                ("m_split", ctypes.c_int32), ("workspace", ctypes.c_int64),
                ("source", ctypes.c_int32), ("tail_variant", ctypes.c_char * 48),
                ("tail_split_k", ctypes.c_int32)]


def load():
    """Load the in-tree libbsmm.so (once) and declare its prototypes.

    PyTorch is imported first: its HIP runtime must be the one in the
    process before the library's own dependency on a HIP runtime is
    resolved, or the library would bring in a second runtime whose launches
    and allocations do not mix with torch's.
    """
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(lib_path):
        raise RuntimeError(f"{lib_path} is not built; run __graft_entry__.build()")
    import torch  # noqa: F401  (see above)
    L = ctypes.CDLL(lib_path)
    i64, vp, sz, st = ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    L.bsmm_int8_rowwise.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, st,
                                    i64, i64, i64, vp, sz, vp]
    L.bsmm_fp8_blockwise.argtypes = [vp, i64, vp, i64, vp, i64, i64, vp, i64, i64,
                                     vp, i64, st, i64, i64, i64, vp, sz, vp]
    L.bsmm_fp8_groupwise.argtypes = [vp, i64, vp, i64, vp, i64, i64, vp, i64, i64,
                                     vp, i64, st, i64, i64, i64, vp, sz, vp]
    L.bsmm_fp8_blockwise_scratch.argtypes = [vp, i64, vp, i64, vp, i64, i64, vp, i64, i64,
                                             vp, i64, st, i64, i64, i64, vp]
    L.bsmm_fp8_mx_bmm.argtypes = [vp, i64, i64, vp, i64, i64, vp, i64, i64, vp, i64,
                                  i64, vp, i64, i64, st, i64, i64, i64, i64, vp, sz, vp]
    L.bsmm_fp8_scaled_mm.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, vp, st, vp,
                                     vp, i64, st, i64, i64, i64, vp, sz, vp]
    L.bsmm_fp8_mx32_mm.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, st, i64, i64,
                                   i64, vp, sz, vp]
    L.bsmm_quant_int8_rowwise.argtypes = [vp, i64, st, vp, i64, vp, i64, i64, i64, vp]
    L.bsmm_quant_fp8_blockwise.argtypes = [vp, i64, st, vp, i64, vp, i64, i64, i64, i64, vp]
    L.bsmm_quant_fp8_mx.argtypes = [vp, i64, st, vp, i64, vp, i64, i64, i64, i64, vp]
    L.bsmm_quant_fp8_mx32.argtypes = [vp, i64, st, vp, i64, vp, i64, i64, i64, i64, vp]
    L.bsmm_quant_fp8_columns.argtypes = [vp, i64, st, vp, i64, vp, i64, i64, i64, i64, vp]
    L.bsmm_quant_fp8_weight.argtypes = [vp, i64, st, vp, i64, vp, i64, vp, i64, i64, i64, i64,
                                        vp]
    L.bsmm_quant_fp8_blockwise_columns.argtypes = [vp, i64, st, vp, i64, vp, i64, i64, vp, i64,
                                                   vp, i64, i64, i64, i64, vp]
    L.bsmm_quant_w4.argtypes = [vp, i64, st, vp, i64, vp, i64, st, vp, i64, vp, i64, st, i64,
                                i64, vp]
    L.bsmm_w4_mm.argtypes = [vp, i64, st, vp, i64, vp, i64, st, vp, i64, st, vp, i64, st,
                             i64, i64, i64, vp, sz, vp]
    L.bsmm_w4_expert_mm.argtypes = [vp, i64, st, vp, i64, i64, vp, i64, i64, st, vp, i64, i64, st,
                                    vp, vp, st, vp, vp, i64, st, i64, i64, i64, i64, i64, vp, sz,
                                    vp]
    L.bsmm_expert_mm.argtypes = [vp, i64, vp, i64, i64, i64, st, vp, vp, st, vp, vp, i64, st, i64,
                                 i64, i64, i64, i64, vp, sz, vp]
    L.bsmm_expert_wgrad.argtypes = [vp, i64, st, st, vp, i64, st, vp, i64, vp, vp, vp, i64, i64,
                                    st, i64, i64, i64, i64, i64, i64, vp, sz, vp]
    L.bsmm_expert_mm_workspace_bytes.argtypes = [st, st, i64, i64, i64, i64]
    L.bsmm_expert_mm_workspace_bytes.restype = sz
    L.bsmm_expert_wgrad_workspace_bytes.argtypes = [st, st, i64, i64, i64, i64, i64]
    L.bsmm_expert_wgrad_workspace_bytes.restype = sz
    L.bsmm_expert_mm_plan_name.argtypes = [st, st, st, i64, i64, i64, i64, sz, vp]
    L.bsmm_expert_mm_plan_name.restype = ctypes.c_char_p
    L.bsmm_expert_wgrad_plan_name.argtypes = [st, st, st, st, st, i64, i64, i64, i64, i64, sz,
                                              vp]
    L.bsmm_expert_wgrad_plan_name.restype = ctypes.c_char_p
    L.bsmm_quant_int8_mx.argtypes = [vp, i64, st, vp, i64, vp, i64, vp, i64, i64, i64, vp]
    L.bsmm_swiglu.argtypes = [vp, i64, st, vp, i64, vp, i64, vp, i64, i64, i64, vp]
    L.bsmm_swiglu_backward.argtypes = [vp, i64, st, vp, i64, vp, i64, vp, vp, i64, vp, i64, vp,
                                       i64, i64, vp]
    L.bsmm_w4_workspace_bytes.argtypes = [st, i64, i64, i64, i64, i64, st]
    L.bsmm_w4_workspace_bytes.restype = sz
    L.bsmm_w4_plan_name.argtypes = [st, st, i64, i64, i64, i64, i64, st]
    L.bsmm_w4_plan_name.restype = ctypes.c_char_p
    L.bsmm_route_workspace_bytes.argtypes = [i64, i64]
    L.bsmm_route_workspace_bytes.restype = sz
    L.bsmm_route_topk.argtypes = [vp, i64, st, vp, st, st, ctypes.c_float, vp, vp, vp, vp, vp, vp,
                                  vp, vp, i64, i64, vp, sz, vp]
    L.bsmm_route_topk_backward.argtypes = [vp, i64, st, vp, vp, vp, vp, vp, st, st,
                                           ctypes.c_float, vp, vp, vp, i64, i64, i64, vp]
    for f in ("bsmm_int8_rowwise", "bsmm_fp8_blockwise", "bsmm_fp8_blockwise_scratch",
              "bsmm_fp8_mx_bmm", "bsmm_fp8_scaled_mm",
              "bsmm_fp8_mx32_mm",
              "bsmm_quant_int8_rowwise", "bsmm_quant_fp8_blockwise", "bsmm_quant_fp8_mx",
              "bsmm_quant_fp8_mx32", "bsmm_quant_fp8_columns", "bsmm_quant_fp8_weight",
              "bsmm_quant_fp8_blockwise_columns", "bsmm_quant_w4", "bsmm_w4_mm",
              "bsmm_w4_expert_mm", "bsmm_expert_mm", "bsmm_expert_wgrad", "bsmm_quant_int8_mx",
              "bsmm_swiglu", "bsmm_swiglu_backward", "bsmm_route_topk",
              "bsmm_route_topk_backward"):
        getattr(L, f).restype = st
    L.bsmm_workspace_bytes.argtypes = [st, i64, i64, i64, i64, st]
    L.bsmm_workspace_bytes.restype = sz
    L.bsmm_query_plan.argtypes = [st, i64, i64, i64, i64, st, sz, ctypes.POINTER(PlanInfo)]
    L.bsmm_query_plan.restype = st
    L.bsmm_set_override.argtypes = [ctypes.c_char_p, st]
    L.bsmm_set_override.restype = st
    L.bsmm_set_override_tail.argtypes = [st, ctypes.c_char_p, st]
    L.bsmm_set_override_tail.restype = st
    L.bsmm_set_streamk_grid.argtypes = [st]
    L.bsmm_set_streamk_grid.restype = st
    L.bsmm_mfma_probe.argtypes = [st, st, st, vp, vp]
    L.bsmm_mfma_probe.restype = st
    L.bsmm_variant_names.restype = ctypes.c_char_p
    L.bsmm_status_string.argtypes = [st]
    L.bsmm_status_string.restype = ctypes.c_char_p
    L.bsmm_last_error.restype = ctypes.c_char_p
    L.bsmm_version.restype = st
    L.bsmm_timing_enable.argtypes = [ctypes.c_int]
    L.bsmm_timing_enable.restype = st
    L.bsmm_timing_read.argtypes = [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(i64),
                                   ctypes.c_char_p, sz]
    L.bsmm_timing_read.restype = st
    _lib = L
    return L


def _check(status):
    if status != 0:
        raise BsmmError(status, load().bsmm_last_error().decode())


# ----------------------------------------------------------------- helpers --

def _torch():
    import torch
    return torch


_CURRENT = []     # torch's functions for the current device and its current stream


def _stream(stream):
    """The HIP stream handle of ``stream``, or of the current stream of the
    current device (read without building a Stream object: the per-call
    host cost matters for decode-sized calls)."""
    if stream is not None:
        return stream.cuda_stream
    if not _CURRENT:
        torch = _torch()
        torch.cuda.current_device()          # initialises the device once
        get = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        raw = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda device: torch.cuda.current_stream(device).cuda_stream)
        _CURRENT.append((get, raw))
    get, raw = _CURRENT[0]
    return raw(get())


class _Workspaces(threading.local):
    """A host thread's workspaces: (address, bytes) per (device, stream handle)."""

    def __init__(self):
        self.by = {}


_WS = _Workspaces()
_WS_NEED = {}     # workspace bytes per (op, G, M, N, K, out dtype); cleared by the override


class _Address(int):
    """A buffer's address that keeps the buffer alive."""


def _workspace(op, G, M, N, K, out_dtype, device, stream, handle):
    """Workspace for the fastest plan of a GEMM (see _buffer)."""
    key = (op, G, M, N, K, out_dtype)
    need = _WS_NEED.get(key)
    if need is None:
        need = load().bsmm_workspace_bytes(op, G, M, N, K, out_dtype)
        _WS_NEED[key] = need
    return _buffer(need, device, stream, handle)


def _capturing(stream):
    """Whether ``stream`` (None: the current one) is being captured."""
    cuda = _torch().cuda
    if stream is None:
        return cuda.is_current_stream_capturing()
    with cuda.stream(stream):
        return cuda.is_current_stream_capturing()


def _new_buffer(need, device, stream):
    torch = _torch()
    if stream is None:
        buf = torch.empty(need, dtype=torch.uint8, device=device)
    else:
        with torch.cuda.stream(stream):
            buf = torch.empty(need, dtype=torch.uint8, device=device)
    address = _Address(buf.data_ptr())
    address.buffer = buf
    return address, need


def _buffer(need, device, stream, handle):
    """(address, bytes) of a workspace of at least ``need`` bytes, or (None, 0).

    It is cached per host thread, device and stream, and grown when a call
    needs more.  One thread's calls on one stream run in order, so they may
    share a buffer.  Two threads' calls on one stream do not: a call is several
    launches, and between them another thread may queue its own (the C calls
    release the interpreter's lock).  A buffer is allocated while its stream is
    current, so the caching allocator hands its memory to no other stream
    before the work queued on that stream has finished, even once the buffer
    is replaced by a larger one.

    A call that is captured in a graph gets a buffer of its own instead, from
    the graph's memory: the graph keeps the address, uses it at every replay
    and on whatever stream it is replayed, none of which a buffer shared with
    eager calls, or replaced by a larger one, would survive."""
    if need == 0:
        return None, 0
    if _capturing(stream):
        return _new_buffer(need, device, stream)
    wkey = (device, handle)
    ws = _WS.by.get(wkey)
    if ws is None or ws[1] < need:
        ws = _WS.by[wkey] = _new_buffer(need, device, stream)
    return ws


def _dtype_code(dt):
    torch = _torch()
    if isinstance(dt, int) and not isinstance(dt, bool) and dt in (I32, F32, BF16, E4M3):
        return dt
    if dt in (torch.int32, "i32"):
        return I32
    if dt in (torch.float32, "f32"):
        return F32
    if dt in (torch.bfloat16, "bf16"):
        return BF16
    if dt in (torch.float8_e4m3fn, "e4m3"):
        return E4M3
    raise ValueError(f"unsupported output dtype {dt}")


def _torch_dtype(code):
    torch = _torch()
    return {I32: torch.int32, F32: torch.float32, BF16: torch.bfloat16,
            E4M3: torch.float8_e4m3fn}[code]


def _bytes_view(t, name):
    torch = _torch()
    if t.dtype in (torch.int8, torch.uint8):
        return t
    if t.dtype in (torch.float8_e4m3fn, torch.float8_e8m0fnu):
        return t.view(torch.uint8)
    raise ValueError(f"{name}: expected 1-byte codes, got {t.dtype}")


def _out(out, shape, code, device):
    torch = _torch()
    dt = _torch_dtype(code)
    if out is None:
        return torch.empty(shape, dtype=dt, device=device)
    if tuple(out.shape) != tuple(shape) or out.dtype != dt:
        raise ValueError(f"out must be {tuple(shape)} {dt}, got {tuple(out.shape)} {out.dtype}")
    return out


def _ws_args(workspace, op, G, M, N, K, code, device, stream, handle):
    if workspace is None:
        return _workspace(op, G, M, N, K, code, device, stream, handle)
    return _given(workspace)


def _given(workspace):
    """Pointer and bytes of a caller's workspace (False: none)."""
    if workspace is False:
        return None, 0
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


# ------------------------------------------------------------ entry points --

def bsmm_int8_rowwise(a, b, scale_a=None, scale_b=None, *, out_dtype="bf16",
                      out=None, workspace=None, stream=None):
    """int8 rowwise scaled matmul.

    a: int8 [M, K] with unit stride along K.  b: int8 [K, N] column-major
    (b.stride(0) == 1), e.g. ``b_nk.t()``.  scale_a: fp32 [M, 1] / [M] or a
    0-d scalar (tensorwise); scale_b: fp32 [1, N] / [N] or 0-d.  out_dtype
    "i32" returns the raw int32 accumulators and ignores the scales.
    """
    torch = _torch()
    code = _dtype_code(out_dtype)
    if a.dim() != 2 or b.dim() != 2:
        raise ValueError("a and b must be 2-D")
    M, K = a.shape
    K2, N = b.shape
    if K != K2:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    if a.dtype != torch.int8 or b.dtype != torch.int8:
        raise ValueError("a and b must be int8")
    if K and a.stride(1) != 1:
        raise ValueError(f"a must be row-major, got stride {a.stride()}")
    if K and b.stride(0) != 1:
        raise ValueError(f"b must be column-major, got stride {b.stride()}")
    sa_m = sb_n = 0
    if code != I32:
        if scale_a is None or scale_b is None:
            raise ValueError("scale_a and scale_b are required unless out_dtype is int32")
        if scale_a.dtype != torch.float32 or scale_b.dtype != torch.float32:
            raise ValueError("scales must be fp32")
        if scale_a.dim() == 0 and scale_b.dim() == 0:
            pass                                     # tensorwise
        elif (tuple(scale_a.shape) in ((M, 1), (M,)) and tuple(scale_b.shape) in ((1, N), (N,))):
            sa_m = scale_a.stride(0)
            sb_n = scale_b.stride(-1)
        else:
            raise ValueError(
                "Invalid scaling configuration. For tensorwise scaling, both scales "
                f"should be scalar. For rowwise scaling, scale_a should be ({M}, 1), "
                f"scale_b should be (1, {N}). Got scale_a.size()={tuple(scale_a.shape)} "
                f"and scale_b.size()={tuple(scale_b.shape)}")
    o = _out(out, (M, N), code, a.device)
    hs = _stream(stream)
    wsp, wsn = _ws_args(workspace, OP_INT8_ROWWISE, 1, M, N, K, code, a.device, stream, hs)
    _check(load().bsmm_int8_rowwise(
        a.data_ptr(), a.stride(0), b.data_ptr(), b.stride(1),
        scale_a.data_ptr() if scale_a is not None else None, sa_m,
        scale_b.data_ptr() if scale_b is not None else None, sb_n,
        o.data_ptr(), o.stride(0), code, M, N, K, wsp, wsn, hs))
    return o


def bsmm_fp8_blockwise(a, b, scale_a, scale_b, *, out_dtype="bf16", out=None,
                       workspace=None, stream=None):
    """fp8 E4M3 blockwise scaled matmul.

    a: [M, K] E4M3 codes (float8_e4m3fn or uint8), row-major.  b: [K, N]
    column-major.  scale_a: fp32 [M, K/128]; scale_b: fp32 [K/128, N/128]
    (any strides).
    """
    torch = _torch()
    code = _dtype_code(out_dtype)
    a8, b8 = _bytes_view(a, "a"), _bytes_view(b, "b")
    M, K = a8.shape
    K2, N = b8.shape
    if K != K2:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    if K and a8.stride(1) != 1:
        raise ValueError(f"a must be row-major, got stride {a8.stride()}")
    if K and b8.stride(0) != 1:
        raise ValueError(f"b must be column-major, got stride {b8.stride()}")
    KB, NB = -(-K // 128), -(-N // 128)
    if scale_a.dtype != torch.float32 or scale_b.dtype != torch.float32:
        raise ValueError("blockwise scales must be fp32")
    if tuple(scale_a.shape) != (M, KB) or tuple(scale_b.shape) != (KB, NB):
        raise ValueError(
            "Invalid scaling configuration. For blockwise scaling, scale_a should be "
            f"({M}, {KB}) and scale_b should be ({KB}, {NB}). Got "
            f"scale_a.size()={tuple(scale_a.shape)} and scale_b.size()={tuple(scale_b.shape)}")
    o = _out(out, (M, N), code, a8.device)
    hs = _stream(stream)
    wsp, wsn = _ws_args(workspace, OP_FP8_BLOCKWISE, 1, M, N, K, code, a8.device, stream, hs)
    _check(load().bsmm_fp8_blockwise(
        a8.data_ptr(), a8.stride(0), b8.data_ptr(), b8.stride(1),
        scale_a.data_ptr(), scale_a.stride(0), scale_a.stride(1),
        scale_b.data_ptr(), scale_b.stride(0), scale_b.stride(1),
        o.data_ptr(), o.stride(0), code, M, N, K, wsp, wsn, hs))
    return o


def bsmm_fp8_blockwise_scratch(a, b, scale_a, scale_b, *, out_dtype="bf16", out=None,
                               stream=None):
    """bsmm_fp8_blockwise with the library's static device scratch as its
    workspace: the library allocates nothing (pass ``out`` to allocate
    nothing here either).  Same arguments and results; problems whose plan
    needs more than the scratch holds raise BsmmError (BSMM_ERR_UNSUPPORTED).
    Calls that overlap on one GPU race on its scratch."""
    torch = _torch()
    code = _dtype_code(out_dtype)
    a8, b8 = _bytes_view(a, "a"), _bytes_view(b, "b")
    M, K = a8.shape
    K2, N = b8.shape
    if K != K2:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    if K and a8.stride(1) != 1:
        raise ValueError(f"a must be row-major, got stride {a8.stride()}")
    if K and b8.stride(0) != 1:
        raise ValueError(f"b must be column-major, got stride {b8.stride()}")
    KB, NB = -(-K // 128), -(-N // 128)
    if scale_a.dtype != torch.float32 or scale_b.dtype != torch.float32:
        raise ValueError("blockwise scales must be fp32")
    if tuple(scale_a.shape) != (M, KB) or tuple(scale_b.shape) != (KB, NB):
        raise ValueError(
            "Invalid scaling configuration. For blockwise scaling, scale_a should be "
            f"({M}, {KB}) and scale_b should be ({KB}, {NB}). Got "
            f"scale_a.size()={tuple(scale_a.shape)} and scale_b.size()={tuple(scale_b.shape)}")
    o = _out(out, (M, N), code, a8.device)
    _check(load().bsmm_fp8_blockwise_scratch(
        a8.data_ptr(), a8.stride(0), b8.data_ptr(), b8.stride(1),
        scale_a.data_ptr(), scale_a.stride(0), scale_a.stride(1),
        scale_b.data_ptr(), scale_b.stride(0), scale_b.stride(1),
        o.data_ptr(), o.stride(0), code, M, N, K, _stream(stream)))
    return o


def bsmm_fp8_groupwise(a, b, scale_a, scale_b, *, out_dtype="bf16", out=None,
                       workspace=None, stream=None):
    """fp8 E4M3 matmul with 1 x 128 groups on both operands (the weight
    gradient of a blockwise fp8 linear layer).

    a: [M, K] E4M3 codes, row-major.  b: [K, N] column-major.  scale_a: fp32
    [M, K/128] (per row of a and K block); scale_b: fp32 [K/128, N] (per K
    block and column of b); any strides.  The call needs a workspace (the
    default allocates one); ``workspace=False`` is rejected by the library.
    """
    torch = _torch()
    code = _dtype_code(out_dtype)
    a8, b8 = _bytes_view(a, "a"), _bytes_view(b, "b")
    M, K = a8.shape
    K2, N = b8.shape
    if K != K2:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    if K and a8.stride(1) != 1:
        raise ValueError(f"a must be row-major, got stride {a8.stride()}")
    if K and b8.stride(0) != 1:
        raise ValueError(f"b must be column-major, got stride {b8.stride()}")
    KB = -(-K // 128)
    if scale_a.dtype != torch.float32 or scale_b.dtype != torch.float32:
        raise ValueError("groupwise scales must be fp32")
    if tuple(scale_a.shape) != (M, KB) or tuple(scale_b.shape) != (KB, N):
        raise ValueError(
            "Invalid scaling configuration. For groupwise (1x128 x 128x1) scaling, scale_a "
            f"should be ({M}, {KB}) and scale_b should be ({KB}, {N}). Got "
            f"scale_a.size()={tuple(scale_a.shape)} and scale_b.size()={tuple(scale_b.shape)}")
    o = _out(out, (M, N), code, a8.device)
    hs = _stream(stream)
    wsp, wsn = _ws_args(workspace, OP_FP8_GROUPWISE, 1, M, N, K, code, a8.device, stream, hs)
    _check(load().bsmm_fp8_groupwise(
        a8.data_ptr(), a8.stride(0), b8.data_ptr(), b8.stride(1),
        scale_a.data_ptr(), scale_a.stride(0), scale_a.stride(1),
        scale_b.data_ptr(), scale_b.stride(0), scale_b.stride(1),
        o.data_ptr(), o.stride(0), code, M, N, K, wsp, wsn, hs))
    return o


def bsmm_fp8_mx_bmm(x, w, x_scale, w_scale, *, layout="m_major", out_dtype="bf16",
                    out=None, workspace=None, stream=None):
    """fp8 E4M3 batched matmul with e8m0 per-128-K-block scales.

    layout "m_major": x [M, G, K], x_scale [M, G, K/128], out [M, G, N].
    layout "batch_first": x [G, M, K], x_scale [G, M, K/128], out [G, M, N].
    w [G, N, K] and w_scale [G, N/128, K/128] in both.  Arbitrary strides
    with unit stride along K.
    """
    code = _dtype_code(out_dtype)
    x8, w8 = _bytes_view(x, "x"), _bytes_view(w, "w")
    xs8, ws8 = _bytes_view(x_scale, "x_scale"), _bytes_view(w_scale, "w_scale")
    if x8.dim() != 3 or w8.dim() != 3:
        raise ValueError("x and w must be 3-D")
    if layout == "m_major":
        M, G, K = x8.shape
        x_sg, x_sm = x8.stride(1), x8.stride(0)
    elif layout == "batch_first":
        G, M, K = x8.shape
        x_sg, x_sm = x8.stride(0), x8.stride(1)
    else:
        raise ValueError(f"unknown layout {layout}")
    G2, N, K2 = w8.shape
    if G2 != G or K2 != K:
        raise ValueError(f"x {tuple(x8.shape)} and w {tuple(w8.shape)} disagree")
    if K and (x8.stride(2) != 1 or w8.stride(2) != 1):
        raise ValueError("x and w must be contiguous along K")
    KB, NB = -(-K // 128), -(-N // 128)
    want_xs = (M, G, KB) if layout == "m_major" else (G, M, KB)
    if tuple(xs8.shape) != want_xs or tuple(ws8.shape) != (G, NB, KB):
        raise ValueError(
            f"Invalid scaling configuration. For mxscale BMM ({layout}), x_scale should be "
            f"{want_xs} and w_scale should be {(G, NB, KB)}. Got x_scale.size()="
            f"{tuple(xs8.shape)} and w_scale.size()={tuple(ws8.shape)}")
    if KB and (xs8.stride(2) != 1 or ws8.stride(2) != 1):
        raise ValueError("scales must be contiguous along K/128")
    if layout == "m_major":
        xs_sg, xs_sm = xs8.stride(1), xs8.stride(0)
        oshape = (M, G, N)
    else:
        xs_sg, xs_sm = xs8.stride(0), xs8.stride(1)
        oshape = (G, M, N)
    o = _out(out, oshape, code, x8.device)
    if layout == "m_major":
        o_sg, o_sm = o.stride(1), o.stride(0)
    else:
        o_sg, o_sm = o.stride(0), o.stride(1)
    if o.stride(2) != 1:
        raise ValueError("out must be contiguous along N")
    hs = _stream(stream)
    wsp, wsn = _ws_args(workspace, OP_FP8_MX_BMM, G, M, N, K, code, x8.device, stream, hs)
    _check(load().bsmm_fp8_mx_bmm(
        x8.data_ptr(), x_sg, x_sm, w8.data_ptr(), w8.stride(0), w8.stride(1),
        xs8.data_ptr(), xs_sg, xs_sm, ws8.data_ptr(), ws8.stride(0), ws8.stride(1),
        o.data_ptr(), o_sg, o_sm, code, G, M, N, K, wsp, wsn, hs))
    return o


def bsmm_fp8_scaled_mm(a, b, scale_a, scale_b, *, bias=None, scale_result=None,
                       out_dtype="bf16", out=None, workspace=None, stream=None):
    """fp8 E4M3 scaled matmul with tensorwise or rowwise fp32 scales.

    a: [M, K] E4M3 codes, row-major; b: [K, N] column-major.  Tensorwise:
    scale_a and scale_b one element each (shape () or (1, 1)); rowwise:
    scale_a (M, 1), scale_b (1, N).  bias: optional [N] fp32 or bf16.
    scale_result: optional one-element fp32 tensor (or a float).  out_dtype:
    "f32", "bf16" or "e4m3" (torch.float8_e4m3fn).
    """
    torch = _torch()
    code = _dtype_code(out_dtype)
    if code == I32:
        raise ValueError("fp8 scaled_mm writes f32, bf16 or e4m3")
    a8, b8 = _bytes_view(a, "a"), _bytes_view(b, "b")
    M, K = a8.shape
    K2, N = b8.shape
    if K != K2:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    if K and a8.stride(1) != 1:
        raise ValueError(f"a must be row-major, got stride {a8.stride()}")
    if K and b8.stride(0) != 1:
        raise ValueError(f"b must be column-major, got stride {b8.stride()}")
    if scale_a.dtype != torch.float32 or scale_b.dtype != torch.float32:
        raise ValueError("scale_a and scale_b must be fp32")
    if scale_a.numel() == 1 and scale_b.numel() == 1:      # tensorwise: one value each
        sa_m, sb_n = 0, 0
    elif tuple(scale_a.shape) == (M, 1) and tuple(scale_b.shape) == (1, N):
        sa_m, sb_n = scale_a.stride(0), scale_b.stride(1)
    else:
        raise ValueError(
            f"scale shapes: tensorwise takes two scalars, rowwise scale_a ({M}, 1) and "
            f"scale_b (1, {N}); got {tuple(scale_a.shape)} and {tuple(scale_b.shape)}")
    bias_ptr, bias_code = None, F32
    if bias is not None:
        if bias.dtype not in (torch.float32, torch.bfloat16) or bias.dim() != 1 or \
                bias.shape[0] != N or (N and bias.stride(0) != 1):
            raise ValueError(f"bias must be a contiguous [N={N}] fp32 or bf16 tensor")
        bias_ptr, bias_code = bias.data_ptr(), _dtype_code(bias.dtype)
    sr_ptr = None
    if scale_result is not None:
        if not isinstance(scale_result, torch.Tensor):
            scale_result = torch.tensor([float(scale_result)], dtype=torch.float32,
                                        device=a8.device)
        if scale_result.dtype != torch.float32 or scale_result.numel() != 1:
            raise ValueError("scale_result must be one fp32 value")
        sr_ptr = scale_result.data_ptr()
    o = _out(out, (M, N), code, a8.device)
    o8 = o.view(torch.uint8) if code == E4M3 else o
    hs = _stream(stream)
    wsp, wsn = _ws_args(workspace, OP_FP8_SCALED_MM, 1, M, N, K, code, a8.device, stream, hs)
    _check(load().bsmm_fp8_scaled_mm(
        a8.data_ptr(), a8.stride(0), b8.data_ptr(), b8.stride(1),
        scale_a.data_ptr(), sa_m, scale_b.data_ptr(), sb_n, bias_ptr, bias_code, sr_ptr,
        o8.data_ptr(), o.stride(0), code, M, N, K, wsp, wsn, hs))
    return o


def bsmm_fp8_mx32_mm(a, b, a_scale, b_scale, *, out_dtype="bf16", out=None, workspace=None,
                     stream=None):
    """fp8 E4M3 matmul with e8m0 scales on 32-element K blocks (MX).

    a: [M, K] E4M3 codes, row-major; b: [K, N] column-major; a_scale
    [M, K/32] and b_scale [N, K/32] e8m0 bytes (uint8 or float8_e8m0fnu)
    with contiguous rows.
    """
    code = _dtype_code(out_dtype)
    if code not in (F32, BF16):
        raise ValueError("fp8 mx32 writes f32 or bf16")
    a8, b8 = _bytes_view(a, "a"), _bytes_view(b, "b")
    sa8, sb8 = _bytes_view(a_scale, "a_scale"), _bytes_view(b_scale, "b_scale")
    M, K = a8.shape
    K2, N = b8.shape
    if K != K2:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    if K and a8.stride(1) != 1:
        raise ValueError(f"a must be row-major, got stride {a8.stride()}")
    if K and b8.stride(0) != 1:
        raise ValueError(f"b must be column-major, got stride {b8.stride()}")
    KC = -(-K // 32)
    if tuple(sa8.shape) != (M, KC) or tuple(sb8.shape) != (N, KC):
        raise ValueError(f"MX scales: a_scale should be ({M}, {KC}) and b_scale ({N}, {KC}); "
                         f"got {tuple(sa8.shape)} and {tuple(sb8.shape)}")
    if KC and (sa8.stride(1) != 1 or sb8.stride(1) != 1):
        raise ValueError("scale rows must be contiguous")
    o = _out(out, (M, N), code, a8.device)
    hs = _stream(stream)
    wsp, wsn = _ws_args(workspace, OP_FP8_MX32_MM, 1, M, N, K, code, a8.device, stream, hs)
    _check(load().bsmm_fp8_mx32_mm(
        a8.data_ptr(), a8.stride(0), b8.data_ptr(), b8.stride(1),
        sa8.data_ptr(), sa8.stride(0), sb8.data_ptr(), sb8.stride(0),
        o.data_ptr(), o.stride(0), code, M, N, K, wsp, wsn, hs))
    return o


def _quant_input(x, name="x"):
    """A bf16 / fp32 tensor as rows of K: (rows view, input dtype code)."""
    torch = _torch()
    if x.dtype == torch.bfloat16:
        code = BF16
    elif x.dtype == torch.float32:
        code = F32
    else:
        raise ValueError(f"{name}: expected bf16 or fp32, got {x.dtype}")
    if x.dim() < 2:
        raise ValueError(f"{name} must have at least 2 dimensions")
    K = x.shape[-1]
    if K and x.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous along its last dimension")
    if x.dim() == 2:
        return x, code
    if K == 0:
        n = 1
        for d in x.shape[:-1]:
            n *= d
        return x.new_empty((n, 0)), code
    try:
        rows = x.view(-1, K)
    except RuntimeError as e:
        raise ValueError(f"{name}: leading dimensions do not form rows of one stride") from e
    return rows, code


def _quant_out(t, shape, dtype, name, device):
    torch = _torch()
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype:
        raise ValueError(f"{name} must be {tuple(shape)} {dtype}, got {tuple(t.shape)} {t.dtype}")
    return t


def bsmm_quant_int8_rowwise(x, *, q=None, scale=None, stream=None):
    """Per-row symmetric int8 quantisation of x [M, K] (bf16 or fp32).

    Returns (q int8 [M, K], scale fp32 [M, 1]) with x ~ q * scale: the
    operand and scale_a of bsmm_int8_rowwise.
    """
    torch = _torch()
    x2, code = _quant_input(x)
    if x.dim() != 2:
        raise ValueError("x must be 2-D [M, K]")
    M, K = x2.shape
    q = _quant_out(q, (M, K), torch.int8, "q", x.device)
    scale = _quant_out(scale, (M, 1), torch.float32, "scale", x.device)
    if K and q.stride(1) != 1:
        raise ValueError("q must be row-major")
    _check(load().bsmm_quant_int8_rowwise(
        x2.data_ptr(), x2.stride(0), code, q.data_ptr(), q.stride(0),
        scale.data_ptr(), scale.stride(0), M, K, _stream(stream)))
    return q, scale


def bsmm_quant_fp8_blockwise(x, *, q=None, scale=None, stream=None):
    """fp8 E4M3 quantisation of x [M, K] with one fp32 scale per 1 x 128 block.

    Returns (q float8_e4m3fn [M, K], scale fp32 [M, K/128]); a given
    ``scale`` may have any strides (e.g. the column-major transpose).
    """
    torch = _torch()
    x2, code = _quant_input(x)
    if x.dim() != 2:
        raise ValueError("x must be 2-D [M, K]")
    M, K = x2.shape
    KB = K // 128
    q = _quant_out(q, (M, K), torch.float8_e4m3fn, "q", x.device)
    scale = _quant_out(scale, (M, KB), torch.float32, "scale", x.device)
    if K and q.stride(1) != 1:
        raise ValueError("q must be row-major")
    q8 = q.view(torch.uint8)
    _check(load().bsmm_quant_fp8_blockwise(
        x2.data_ptr(), x2.stride(0), code, q8.data_ptr(), q8.stride(0),
        scale.data_ptr(), scale.stride(0), scale.stride(1), M, K, _stream(stream)))
    return q, scale


def bsmm_quant_fp8_columns(x, *, q_t=None, scale=None, stream=None):
    """fp8 E4M3 quantisation of x [R, C] (bf16 or fp32; R a multiple of 128,
    C of 8) in groups of 128 consecutive rows of one column, one fp32 scale
    each: the operands of the weight-gradient GEMM bsmm_fp8_groupwise, which
    contracts over the R tokens.

    Returns (q_t float8_e4m3fn [C, R], the codes transposed, and scale fp32
    [R/128, C]).  With dY [R, N] and X [R, K] quantised this way,
    ``bsmm_fp8_groupwise(dYq_t, Xq_t.t(), s_dy.t(), s_x)`` is dW [N, K].
    """
    torch = _torch()
    x2, code = _quant_input(x)
    if x.dim() != 2:
        raise ValueError("x must be 2-D [R, C]")
    R, C = x2.shape
    q_t = _quant_out(q_t, (C, R), torch.float8_e4m3fn, "q_t", x.device)
    scale = _quant_out(scale, (R // 128, C), torch.float32, "scale", x.device)
    if R and q_t.stride(1) != 1:
        raise ValueError("q_t must be row-major")
    q8 = q_t.view(torch.uint8)
    _check(load().bsmm_quant_fp8_columns(
        x2.data_ptr(), x2.stride(0), code, q8.data_ptr(), q8.stride(0),
        scale.data_ptr(), scale.stride(0), scale.stride(1), R, C, _stream(stream)))
    return q_t, scale


def bsmm_quant_fp8_blockwise_columns(x, *, q=None, scale=None, q_t=None, scale_t=None,
                                     stream=None):
    """Both fp8 quantisations of a layer input x [R, C] (bf16 or fp32; R and C
    multiples of 128) from one read of x: the 1 x 128 row blocks of
    bsmm_quant_fp8_blockwise (the forward GEMM's A) and the groups of 128
    rows down the columns of bsmm_quant_fp8_columns (the weight gradient's
    operand).  Bit-identical to the two separate calls.

    Returns (q float8_e4m3fn [R, C], scale fp32 [R, C/128], q_t
    float8_e4m3fn [C, R], scale_t fp32 [R/128, C]).  Unless given, ``scale``
    is allocated column-major (strides (1, R)): the kernel writes one
    128-column block of every row per tile, which is then one contiguous
    run; bsmm_fp8_blockwise takes scale_a with any strides.
    """
    torch = _torch()
    x2, code = _quant_input(x)
    if x.dim() != 2:
        raise ValueError("x must be 2-D [R, C]")
    R, C = x2.shape
    q = _quant_out(q, (R, C), torch.float8_e4m3fn, "q", x.device)
    if scale is None:
        scale = torch.empty((C // 128, R), dtype=torch.float32, device=x.device).t()
    scale = _quant_out(scale, (R, C // 128), torch.float32, "scale", x.device)
    q_t = _quant_out(q_t, (C, R), torch.float8_e4m3fn, "q_t", x.device)
    scale_t = _quant_out(scale_t, (R // 128, C), torch.float32, "scale_t", x.device)
    for t, n in ((q, "q"), (q_t, "q_t")):
        if t.numel() and t.stride(1) != 1:
            raise ValueError(f"{n} must be row-major")
    qv, qtv = q.view(torch.uint8), q_t.view(torch.uint8)
    _check(load().bsmm_quant_fp8_blockwise_columns(
        x2.data_ptr(), x2.stride(0), code, qv.data_ptr(), qv.stride(0),
        scale.data_ptr(), scale.stride(0), scale.stride(1), qtv.data_ptr(), qtv.stride(0),
        scale_t.data_ptr(), scale_t.stride(0), scale_t.stride(1), R, C, _stream(stream)))
    return q, scale, q_t, scale_t


def bsmm_quant_fp8_weight(w, *, plain=True, transposed=True, q=None, q_t=None, scale=None,
                          stream=None):
    """fp8 E4M3 quantisation of a weight w [R, C] (bf16 or fp32; R and C
    multiples of 128) in 128 x 128 blocks, one fp32 scale each.

    Returns (q [R, C] or None, q_t [C, R] or None, scale fp32 [R/128, C/128]):
    the codes as they are (the forward GEMM's B = ``q.t()`` with scale_b
    ``scale.t()``) and transposed (the input gradient's B = ``q_t.t()`` with
    scale_b ``scale``).
    """
    torch = _torch()
    if not (plain or transposed):
        raise ValueError("ask for the plain or the transposed codes (or both)")
    w2, code = _quant_input(w, "w")
    if w.dim() != 2:
        raise ValueError("w must be 2-D [R, C]")
    R, C = w2.shape
    q = _quant_out(q, (R, C), torch.float8_e4m3fn, "q", w.device) if plain else None
    q_t = _quant_out(q_t, (C, R), torch.float8_e4m3fn, "q_t", w.device) if transposed else None
    scale = _quant_out(scale, (R // 128, C // 128), torch.float32, "scale", w.device)
    for t, n in ((q, "q"), (q_t, "q_t")):
        if t is not None and t.numel() and t.stride(1) != 1:
            raise ValueError(f"{n} must be row-major")
    qv = q.view(torch.uint8) if q is not None else None
    qtv = q_t.view(torch.uint8) if q_t is not None else None
    _check(load().bsmm_quant_fp8_weight(
        w2.data_ptr(), w2.stride(0), code,
        qv.data_ptr() if qv is not None else None, qv.stride(0) if qv is not None else 0,
        qtv.data_ptr() if qtv is not None else None, qtv.stride(0) if qtv is not None else 0,
        scale.data_ptr(), scale.stride(0), scale.stride(1), R, C, _stream(stream)))
    return q, q_t, scale


def bsmm_quant_fp8_mx(x, *, block=128, q=None, scale=None, stream=None):
    """fp8 E4M3 quantisation with an e8m0 scale per 1 x ``block`` block
    (128, or 32 for bsmm_fp8_mx32_mm) along the last dimension of x [..., K]
    (bf16 or fp32), e.g. the BMM's x [M, G, K] or [G, M, K].

    Returns (q float8_e4m3fn [..., K], scale uint8 e8m0 bytes
    [..., K/block]): the x and x_scale of bsmm_fp8_mx_bmm, or (block 32) an
    operand and its scales for bsmm_fp8_mx32_mm.
    """
    torch = _torch()
    if block not in (32, 128):
        raise ValueError("block must be 32 or 128")
    x2, code = _quant_input(x)
    K = x.shape[-1]
    lead = tuple(x.shape[:-1])
    q = _quant_out(q, lead + (K,), torch.float8_e4m3fn, "q", x.device)
    scale = _quant_out(scale, lead + (K // block,), torch.uint8, "scale", x.device)
    if not q.is_contiguous() or not scale.is_contiguous():
        raise ValueError("q and scale must be contiguous")
    q8 = q.view(torch.uint8).view(-1, K) if K else q.view(torch.uint8)
    M = x2.shape[0]
    fn = load().bsmm_quant_fp8_mx if block == 128 else load().bsmm_quant_fp8_mx32
    _check(fn(x2.data_ptr(), x2.stride(0), code, q8.data_ptr(), K,
              scale.data_ptr(), K // block, 1, M, K, _stream(stream)))
    return q, scale


def bsmm_quant_w4(w, *, group=128, symmetric=True, scale_dtype="f32", values=False, stream=None):
    """4-bit quantisation of a weight w [..., K] (bf16 or fp32; at least two
    dimensions) with one scale, and unless ``symmetric`` one zero point, per
    ``group`` (32, 64 or 128) elements of a row.

    Returns (q uint8 [..., K/2], scale [..., K/group] of ``scale_dtype``,
    zero uint8 [..., K/group] or None): the operands of bsmm_w4_mm ([N, K])
    and bsmm_w4_expert_mm ([E, N, K]).  ``values=True`` appends what the
    codes stand for, (code - zero) * scale, as a tensor like w.
    """
    w2, code = _quant_input(w, "w")
    sc = _float_code(scale_dtype, "scale_dtype")
    _, torch, dtypes, u8, _, _ = _DTYPES
    if group not in (32, 64, 128):
        raise ValueError("group must be 32, 64 or 128")
    R, K = w2.shape
    if K % group:
        raise ValueError(f"the last dimension ({K}) must be a multiple of group ({group})")
    _one_gpu("w", w)
    lead, dev, KG = w.shape[:-1], w.device, K // group

    def new(cols, dtype):
        if len(lead) == 1:            # the cheapest allocation on the host
            return torch.empty_strided((R, cols), (cols, 1), dtype=dtype, device=dev)
        return torch.empty((*lead, cols), dtype=dtype, device=dev)

    q = new(K // 2, u8)
    scale = new(KG, dtypes[sc])
    zero = None if symmetric else new(KG, u8)
    v = new(K, w.dtype) if values else None
    _check(load().bsmm_quant_w4(
        w2.data_ptr(), w2.stride(0) if R > 1 else K, code, q.data_ptr(), K // 2,
        scale.data_ptr(), KG, sc, None if symmetric else zero.data_ptr(), KG,
        v.data_ptr() if values else None, K, group, R, K, _stream(stream)))
    return (q, scale, zero, v) if values else (q, scale, zero)


_DTYPES = ()      # what _float_types returns (made once)


def _float_types():
    """(library code by torch dtype, name and code of the float dtypes, torch,
    torch dtype by code, uint8, int32, float32)."""
    global _DTYPES
    if not _DTYPES:
        torch = _torch()
        # assigned whole: another thread sees all of it or nothing
        _DTYPES = ({torch.bfloat16: BF16, torch.float32: F32, "bf16": BF16, "f32": F32,
                    BF16: BF16, F32: F32}, torch, {BF16: torch.bfloat16, F32: torch.float32},
                   torch.uint8, torch.int32, torch.float32)
    return _DTYPES


def _float_code(dt, name):
    """F32 or BF16 for a float tensor's dtype."""
    code = _float_types()[0].get(dt)
    if code is None:
        raise ValueError(f"{name}: expected bf16 or fp32, got {dt}")
    return code


def _one_gpu(names, first, *others):
    """Check that the tensors given (None: not given) are all on one GPU: a
    kernel that reads a host address faults."""
    gpu = first.get_device()
    if gpu >= 0:
        for t in others:
            if t is not None and t.get_device() != gpu:
                break
        else:
            return
    raise ValueError(f"{names} must be on one GPU, got " + ", ".join(
        "none" if t is None else str(t.device) for t in (first, *others)))


def _w4_weight(w, ws, wst, scale, zero, K, u8):
    """Check a 4-bit weight (shape ws, strides wst) against K input features;
    returns (group, row stride, scale dtype code, scale strides, zero pointer,
    zero strides), strides as (of the expert, of the row).  The stride of a
    dimension of one element says nothing: a row's length stands for it.  A
    decode call is bound by the host: one read of each shape and stride."""
    code = _float_code(scale.dtype, "scale")
    if w.dtype is not u8 or 2 * ws[-1] != K:
        raise ValueError(f"w must be uint8 with {K // 2} bytes a row (K = {K}), got {w.dtype} "
                         f"{tuple(ws)}")
    ss, sst = scale.shape, scale.stride()
    KG = ss[-1]
    if ss[:-1] != ws[:-1]:
        raise ValueError(f"scale {tuple(ss)} does not fit w {tuple(ws)}")
    if K and (KG == 0 or K % KG):
        raise ValueError(f"scale has {KG} groups for K = {K}")
    if (K and wst[-1] != 1) or (KG > 1 and sst[-1] != 1):
        raise ValueError("w and scale must be contiguous along their last dimension")
    group = K // KG if K else 32
    many = ws[-2] > 1
    ldw = wst[-2] if many else K // 2
    sstride = (sst[0], sst[-2] if many else KG)
    if zero is None:
        return group, ldw, code, sstride, None, (0, 0)
    zst = zero.stride()
    if zero.dtype is not u8 or zero.shape != ss:
        raise ValueError(f"zero must be uint8 {tuple(ss)}, got {zero.dtype} {tuple(zero.shape)}")
    if KG > 1 and zst[-1] != 1:
        raise ValueError("zero must be contiguous along its last dimension")
    return group, ldw, code, sstride, zero.data_ptr(), (zst[0], zst[-2] if many else KG)


def _w4_workspace(workspace, xc, E, R, S, N, K, group, dev, stream, handle):
    """Workspace pointer and bytes of a 4-bit product (fp32 x, many rows)."""
    if workspace is not None:
        return _given(workspace)
    if xc != F32:
        return None, 0
    return _buffer(load().bsmm_w4_workspace_bytes(xc, E, R, S, N, K, group), dev, stream, handle)


def _w4_out(out, rows, cols, code, torch, dtypes, dev):
    """The output tensor [rows, cols] and its row stride."""
    if out is None:
        # the cheapest allocation on the host
        return torch.empty_strided((rows, cols), (cols, 1), dtype=dtypes[code], device=dev), cols
    if tuple(out.shape) != (rows, cols) or out.dtype is not dtypes[code]:
        raise ValueError(f"out must be {(rows, cols)} {dtypes[code]}, got {tuple(out.shape)} "
                         f"{out.dtype}")
    st = out.stride()
    if cols and st[1] != 1:
        raise ValueError("out must be contiguous along its last dimension")
    return out, st[0] if rows > 1 else cols


def bsmm_w4_mm(x, w, scale, zero=None, *, out_dtype="bf16", out=None, workspace=None,
               stream=None):
    """Activations times a 4-bit weight: x @ W.T with W = (code - zero) * scale.

    x: bf16 or fp32 [M, K].  w: uint8 [N, K/2], scale: bf16 or fp32
    [N, K/group], zero: uint8 [N, K/group] or None (8), as bsmm_quant_w4
    returns them (group 32, 64 or 128).  Returns [M, N], fp32 or bf16.
    workspace: None for a cached one, False for none, or a 16-byte aligned
    tensor of bsmm_w4_workspace_bytes bytes.
    """
    xs, ws = x.shape, w.shape
    if len(xs) != 2 or len(ws) != 2:
        raise ValueError("x and w must be 2-D")
    xc = _float_code(x.dtype, "x")
    code = _float_code(out_dtype, "out_dtype")
    _, torch, dtypes, u8, _, _ = _DTYPES
    M, K = xs
    N = ws[0]
    xst, wst = x.stride(), w.stride()
    group, ldw, sc, sst, zp, zst = _w4_weight(w, ws, wst, scale, zero, K, u8)
    if K and xst[1] != 1:
        raise ValueError(f"x must be row-major, got stride {xst}")
    _one_gpu("x, w, scale, zero, out and workspace", x, w, scale, zero, out,
             None if workspace is False else workspace)
    dev = x.device
    o, ldo = _w4_out(out, M, N, code, torch, dtypes, dev)
    hs = _stream(stream)
    wsp, wsn = _w4_workspace(workspace, xc, 1, M, M, N, K, group, dev, stream, hs)
    status = load().bsmm_w4_mm(x.data_ptr(), xst[0] if M > 1 else K, xc, w.data_ptr(), ldw,
                               scale.data_ptr(), sst[1], sc, zp, zst[1], group, o.data_ptr(), ldo,
                               code, M, N, K, wsp, wsn, hs)
    if status:
        _check(status)
    return o


def bsmm_w4_expert_mm(x, w, scale, zero, order, offsets, *, slots_per_row=1, row_scale=None,
                      out_dtype="bf16", out=None, workspace=None, stream=None):
    """Routed rows times their experts' 4-bit weights.

    x: bf16 or fp32 [R, K].  w: uint8 [E, N, K/2], scale [E, N, K/group], zero
    [E, N, K/group] or None, as bsmm_quant_w4 returns them for a weight
    [E, N, K].  order: int32 [S] and offsets: int32 [E + 1] as bsmm_route_topk
    returns them.  Slot s reads row s // slots_per_row of x: slots_per_row is
    the number of choices where x holds tokens, 1 where it holds slots.
    row_scale: fp32 [S] (the routing weights, slot order) or None.  Returns
    [S, N] in slot order, zeros for slots without an expert.  workspace as for
    bsmm_w4_mm.
    """
    xs, ws = x.shape, w.shape
    if len(xs) != 2 or len(ws) != 3:
        raise ValueError("x must be 2-D and w 3-D")
    xc = _float_code(x.dtype, "x")
    code = _float_code(out_dtype, "out_dtype")
    _, torch, dtypes, u8, i32, f32 = _DTYPES
    R, K = xs
    E, N = ws[0], ws[1]
    xst, wst = x.stride(), w.stride()
    group, ldw, sc, sst, zp, zst = _w4_weight(w, ws, wst, scale, zero, K, u8)
    if K and xst[1] != 1:
        raise ValueError(f"x must be row-major, got stride {xst}")
    if order.dtype is not i32 or order.dim() != 1 or not order.is_contiguous():
        raise ValueError("order must be a contiguous int32 [S] tensor")
    S = order.shape[0]
    if offsets.dtype is not i32 or offsets.shape != (E + 1,) or not offsets.is_contiguous():
        raise ValueError(f"offsets must be a contiguous int32 [{E + 1}] tensor")
    if row_scale is not None and (row_scale.dtype is not f32 or row_scale.numel() != S or
                                  not row_scale.is_contiguous()):
        raise ValueError(f"row_scale must be contiguous fp32 of {S} elements")
    _one_gpu("x, w, scale, zero, order, offsets, row_scale, out and workspace", x, w, scale, zero,
             order, offsets, row_scale, out, None if workspace is False else workspace)
    dev = x.device
    o, ldo = _w4_out(out, S, N, code, torch, dtypes, dev)
    hs = _stream(stream)
    wsp, wsn = _w4_workspace(workspace, xc, E, R, S, N, K, group, dev, stream, hs)
    status = load().bsmm_w4_expert_mm(
        x.data_ptr(), xst[0] if R > 1 else K, xc, w.data_ptr(), wst[0] if E > 1 else 0, ldw,
        scale.data_ptr(), sst[0], sst[1], sc, zp, zst[0], zst[1], group, order.data_ptr(),
        offsets.data_ptr(), slots_per_row,
        None if row_scale is None else row_scale.data_ptr(), o.data_ptr(), ldo, code, E, R, S, N,
        K, wsp, wsn, hs)
    if status:
        _check(status)
    return o


def _stream_of(t, stream):
    """_stream, where t is on the device that it belongs to."""
    at = t.get_device()
    if stream is not None:
        if stream.device_index != at:
            raise ValueError(f"tensors on cuda:{at}, but a stream of cuda:{stream.device_index}")
        return stream.cuda_stream
    if not _CURRENT:
        _stream(None)
    get, raw = _CURRENT[0]
    now = get()
    if now != at:
        raise ValueError(f"tensors on cuda:{at}, but the current device is cuda:{now}")
    return raw(now)


def _slots_per_row(n, name):
    if not 1 <= n < 2**31:
        raise ValueError(f"{name} must be at least 1 and below 2^31, got {n}")


def _routed(order, offsets, E, S, i32):
    """Check a Route's order (None: slots as they are) and offsets; returns
    order's address."""
    if order is not None and (order.dtype is not i32 or order.dim() != 1 or
                              order.shape[0] != S or not order.is_contiguous()):
        raise ValueError(f"order must be a contiguous int32 [{S}] tensor")
    if offsets.dtype is not i32 or offsets.shape != (E + 1,) or not offsets.is_contiguous():
        raise ValueError(f"offsets must be a contiguous int32 [{E + 1}] tensor")
    return None if order is None else order.data_ptr()


def _row_stride(t, shape, stride, name):
    """The row stride of a 2-D tensor whose rows are contiguous."""
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D")
    if shape[1] > 1 and stride[1] != 1:
        raise ValueError(f"{name} must be row-major, got stride {stride}")
    return stride[0] if shape[0] > 1 else shape[1]


def bsmm_expert_mm(x, w, order, offsets, *, slots_per_row=1, row_scale=None, out_dtype="bf16",
                   out=None, workspace=None, stream=None):
    """Routed rows times their experts' weights.

    x: bf16 or fp32 [R, K].  w: [E, N, K] of x's type, contiguous along its
    last dimension or its middle one: a weight w [E, N, K] for the product,
    ``w.transpose(1, 2)`` for the gradient of its input from the rows of dy.
    order: int32 [S] and offsets: int32 [E + 1] as bsmm_route_topk returns
    them; order None: the slots are sorted (S = R * slots_per_row).  Slot s
    reads row s // slots_per_row of x.  row_scale: fp32 [S] or None.  Returns
    [S, N] in slot order, zeros for slots without an expert.  workspace: None
    for a cached one, False for none, or a 16-byte aligned tensor of
    bsmm_expert_mm_workspace_bytes bytes.
    """
    xs, ws = x.shape, w.shape
    if len(ws) != 3:
        raise ValueError("w must be 3-D")
    xc = _float_code(x.dtype, "x")
    code = _float_code(out_dtype, "out_dtype")
    _, torch, dtypes, _, i32, f32 = _DTYPES
    ldx = _row_stride(x, xs, x.stride(), "x")
    R, K = xs
    E, N = ws[0], ws[1]
    if w.dtype is not x.dtype or ws[2] != K:
        raise ValueError(f"w must be {x.dtype} with {K} columns, got {w.dtype} {tuple(ws)}")
    # a dimension of one element has no stride to speak of
    se, sn, sk = w.stride()
    if K == 1:
        sk = 1
    elif N == 1 and sk != 1:
        sn = 1
    if K > 1 and N > 1 and sn != 1 and sk != 1:
        raise ValueError(f"w must be contiguous along N or K, got stride {w.stride()}")
    _slots_per_row(slots_per_row, "slots_per_row")
    S = R * slots_per_row if order is None else order.shape[0]
    op = _routed(order, offsets, E, S, i32)
    if row_scale is not None and (row_scale.dtype is not f32 or row_scale.numel() != S or
                                  not row_scale.is_contiguous()):
        raise ValueError(f"row_scale must be contiguous fp32 of {S} elements")
    _one_gpu("x, w, order, offsets, row_scale, out and workspace", x, w, order, offsets, row_scale,
             out, None if workspace is False else workspace)
    o, ldo = _w4_out(out, S, N, code, torch, dtypes, x.device)
    hs = _stream_of(x, stream)
    if workspace is None:
        key = ("expert_mm", xc, sk == 1, E, S, N, K)
        need = _WS_NEED.get(key)
        if need is None:
            need = _WS_NEED[key] = load().bsmm_expert_mm_workspace_bytes(
                xc, 0 if sk == 1 else 1, E, S, N, K)
        wsp, wsn = _buffer(need, x.device, stream, hs)
    else:
        wsp, wsn = _given(workspace)
    status = load().bsmm_expert_mm(
        x.data_ptr(), ldx, w.data_ptr(), se if E > 1 else 0, sn, sk, xc, op, offsets.data_ptr(),
        slots_per_row, None if row_scale is None else row_scale.data_ptr(), o.data_ptr(), ldo,
        code, E, R, S, N, K, wsp, wsn, hs)
    if status:
        _check(status)
    return o


def bsmm_expert_wgrad(dy, x, order, offsets, *, x_scale=None, dy_slots_per_row=1,
                      x_slots_per_row=1, out_dtype="f32", out=None, workspace=None, stream=None):
    """The experts' weight gradients, dw[e] = sum of dy[s]^T x[s] over e's slots.

    dy: bf16 or fp32 [Ry, N].  x: [Rx, K] of dy's type, or with x_scale the
    int8 codes and bytes of bsmm_quant_int8_mx.  Slot s reads row s //
    dy_slots_per_row of dy and s // x_slots_per_row of x.  order: int32 [S] and
    offsets: int32 [E + 1] as bsmm_route_topk returns them; order None: the
    slots are sorted (S = Ry * dy_slots_per_row), and with offsets [0, S] this
    is a dense layer's gradient.  Returns [E, N, K], zeros for experts without
    slots.  workspace: None for a cached one, False for none, or a 16-byte
    aligned tensor of bsmm_expert_wgrad_workspace_bytes bytes.
    """
    yc = _float_code(dy.dtype, "dy")
    code = _float_code(out_dtype, "out_dtype")
    _, torch, dtypes, u8, i32, _ = _DTYPES
    ys, xs = dy.shape, x.shape
    ldy, ldx = _row_stride(dy, ys, dy.stride(), "dy"), _row_stride(x, xs, x.stride(), "x")
    Ry, N = ys
    Rx, K = xs
    sp, s_r = None, 0
    if x_scale is None:
        if x.dtype is not dy.dtype:
            raise ValueError(f"x must be {dy.dtype}, or int8 codes with x_scale; got {x.dtype}")
    else:
        if x.dtype is not torch.int8 or K % 32:
            raise ValueError(f"a checkpoint is int8 with K % 32 == 0, got {x.dtype} {tuple(xs)}")
        ss = x_scale.shape
        if x_scale.dtype is not u8 or ss != (Rx, K // 32):
            raise ValueError(f"x_scale must be uint8 [{Rx}, {K // 32}], got {x_scale.dtype} "
                             f"{tuple(ss)}")
        s_r = _row_stride(x_scale, ss, x_scale.stride(), "x_scale")
        sp = x_scale.data_ptr()
    _slots_per_row(dy_slots_per_row, "dy_slots_per_row")
    _slots_per_row(x_slots_per_row, "x_slots_per_row")
    S = Ry * dy_slots_per_row if order is None else order.shape[0]
    E = offsets.shape[0] - 1 if offsets.dim() == 1 else -1
    if E < 0:
        raise ValueError("offsets must be 1-D [E + 1]")
    op = _routed(order, offsets, E, S, i32)
    _one_gpu("dy, x, x_scale, order, offsets, out and workspace", dy, x, x_scale, order, offsets,
             out, None if workspace is False else workspace)
    if out is None:
        o, se, ldw = torch.empty((E, N, K), dtype=dtypes[code], device=dy.device), N * K, K
    else:
        if tuple(out.shape) != (E, N, K) or out.dtype is not dtypes[code]:
            raise ValueError(f"out must be {(E, N, K)} {dtypes[code]}, got {tuple(out.shape)} "
                             f"{out.dtype}")
        o, (se, ldw, sk) = out, out.stride()
        if K > 1 and sk != 1:
            raise ValueError("out must be contiguous along its last dimension")
        ldw = ldw if N > 1 else K
    hs = _stream_of(dy, stream)
    if workspace is None:
        key = ("expert_wgrad", yc, sp is None, E, Rx, S, N, K)
        need = _WS_NEED.get(key)
        if need is None:
            need = _WS_NEED[key] = load().bsmm_expert_wgrad_workspace_bytes(
                yc, 0 if sp is None else 1, E, Rx, S, N, K)
        wsp, wsn = _buffer(need, dy.device, stream, hs)
    else:
        wsp, wsn = _given(workspace)
    status = load().bsmm_expert_wgrad(
        dy.data_ptr(), ldy, yc, dy_slots_per_row, x.data_ptr(), ldx, x_slots_per_row, sp, s_r, op,
        offsets.data_ptr(), o.data_ptr(), se if E > 1 else 0, ldw, code, E, Ry, Rx, S, N, K, wsp,
        wsn, hs)
    if status:
        _check(status)
    return o


def bsmm_quant_int8_mx(x, *, values=False, stream=None):
    """An 8-bit checkpoint of activations x [..., K] (bf16 or fp32; K a
    multiple of 32): int8 codes and a power of two per 32 elements of a row.

    Returns (q int8 [..., K], scale uint8 e8m0 bytes [..., K/32]), which stand
    for q * 2^(scale - 133): the x of bsmm_expert_wgrad.  ``values=True``
    appends these values as a tensor like x.
    """
    code = _float_code(x.dtype, "x")
    _, torch, _, u8, _, _ = _DTYPES
    xs = x.shape
    x2 = x if len(xs) == 2 else _quant_input(x)[0]
    R, K = x2.shape
    if K % 32:
        raise ValueError(f"the last dimension ({K}) must be a multiple of 32")
    ldx = _row_stride(x2, (R, K), x2.stride(), "x")
    _one_gpu("x", x)
    dev, new = x.device, torch.empty_strided
    q = new((R, K), (K, 1), dtype=torch.int8, device=dev)
    scale = new((R, K // 32), (K // 32, 1), dtype=u8, device=dev)
    v = new((R, K), (K, 1), dtype=x.dtype, device=dev) if values else None
    status = load().bsmm_quant_int8_mx(
        x2.data_ptr(), ldx, code, q.data_ptr(), K, scale.data_ptr(), K // 32,
        v.data_ptr() if values else None, K, R, K, _stream_of(x, stream))
    if status:
        _check(status)
    if x2 is not x:
        q, scale = q.view(xs), scale.view(*xs[:-1], K // 32)
        v = v.view(xs) if values else None
    return (q, scale, v) if values else (q, scale)


def bsmm_swiglu(h, *, checkpoint=False, out=None, stream=None):
    """The gate of a feed-forward layer: silu(h[:, :F]) * h[:, F:].

    h: bf16 or fp32 [R, 2F], F a multiple of 32.  Returns [R, F] of h's type;
    with ``checkpoint`` (that, q int8 [R, 2F], scale uint8 [R, 2F/32]), the
    8-bit checkpoint of h for bsmm_swiglu_backward (as bsmm_quant_int8_mx
    makes it, from the same read).
    """
    code = _float_code(h.dtype, "h")
    _, torch, dtypes, u8, _, _ = _DTYPES
    hs = h.shape
    ldh = _row_stride(h, hs, h.stride(), "h")
    R, F = hs[0], hs[1] // 2
    if hs[1] % 64:
        raise ValueError(f"h must have 2F columns, F a multiple of 32, got {hs[1]}")
    _one_gpu("h and out", h, out)
    dev = h.device
    a, lda = _w4_out(out, R, F, code, torch, dtypes, dev)
    q = scale = None
    if checkpoint:
        q = torch.empty_strided((R, 2 * F), (2 * F, 1), dtype=torch.int8, device=dev)
        scale = torch.empty_strided((R, F // 16), (F // 16, 1), dtype=u8, device=dev)
    status = load().bsmm_swiglu(
        h.data_ptr(), ldh, code, a.data_ptr(), lda, q.data_ptr() if checkpoint else None, 2 * F,
        scale.data_ptr() if checkpoint else None, F // 16, R, F, _stream_of(h, stream))
    if status:
        _check(status)
    return (a, q, scale) if checkpoint else a


def bsmm_swiglu_backward(da, q, scale, *, row_scale=None, act=True, stream=None):
    """The gradient of row_scale * bsmm_swiglu(h) from the checkpoint of h.

    da: bf16 or fp32 [R, F].  q int8 [R, 2F] and scale uint8 [R, 2F/32] as
    bsmm_swiglu returns them.  row_scale: fp32 [R] (the routing weights, where
    they belong to the rows of the gate's output) or None.  Returns (dh
    [R, 2F], act [R, F] = row_scale * the gate's output, both of da's type,
    drow fp32 [R], row_scale's gradient); act and drow are None where ``act``
    is false or row_scale is not given.
    """
    code = _float_code(da.dtype, "da")
    _, torch, _, u8, _, f32 = _DTYPES
    ds = da.shape
    ldda = _row_stride(da, ds, da.stride(), "da")
    R, F = ds
    if F % 32:
        raise ValueError(f"the columns of da ({F}) must be a multiple of 32")
    if q.dtype is not torch.int8 or q.shape != (R, 2 * F):
        raise ValueError(f"q must be int8 [{R}, {2 * F}], got {q.dtype} {tuple(q.shape)}")
    if scale.dtype is not u8 or scale.shape != (R, F // 16):
        raise ValueError(f"scale must be uint8 [{R}, {F // 16}], got {scale.dtype} "
                         f"{tuple(scale.shape)}")
    ldq = _row_stride(q, (R, 2 * F), q.stride(), "q")
    s_r = _row_stride(scale, (R, F // 16), scale.stride(), "scale")
    if row_scale is not None and (row_scale.dtype is not f32 or row_scale.numel() != R or
                                  not row_scale.is_contiguous()):
        raise ValueError(f"row_scale must be contiguous fp32 of {R} elements")
    _one_gpu("da, q, scale and row_scale", da, q, scale, row_scale)
    dev = da.device
    new = torch.empty_strided
    dh = new((R, 2 * F), (2 * F, 1), dtype=da.dtype, device=dev)
    a = new((R, F), (F, 1), dtype=da.dtype, device=dev) if act else None
    drow = None if row_scale is None else new((R,), (1,), dtype=f32, device=dev)
    status = load().bsmm_swiglu_backward(
        da.data_ptr(), ldda, code, q.data_ptr(), ldq, scale.data_ptr(), s_r,
        None if row_scale is None else row_scale.data_ptr(), dh.data_ptr(), 2 * F,
        a.data_ptr() if act else None, F, None if drow is None else drow.data_ptr(), R, F,
        _stream_of(da, stream))
    if status:
        _check(status)
    return dh, a, drow


class Route(NamedTuple):
    """What bsmm_route_topk returns; live, prob_sum and loss are None without
    a loss."""
    index: object        # int32 [T, k]
    weight: object       # fp32 [T, k]
    counts: object       # int32 [E]
    offsets: object      # int32 [E + 1]
    order: object        # int32 [T * k]
    live: object         # int32 [1]
    prob_sum: object     # fp32 [E]
    loss: object         # fp32 [1]


def _route_mask(mask, T):
    torch = _torch()
    if mask is None:
        return None
    if mask.dtype not in (torch.bool, torch.uint8) or tuple(mask.shape) != (T,) or \
            (T > 1 and mask.stride(0) != 1):
        raise ValueError(f"mask must be a contiguous bool or uint8 [{T}] tensor")
    return mask.data_ptr()


def _route_logits(logits):
    """(T, E, row stride, dtype code) of a logits tensor."""
    code = _float_code(logits.dtype, "logits")
    shape, st = logits.shape, logits.stride()
    if len(shape) != 2:
        raise ValueError("logits must be 2-D [T, E]")
    if shape[1] and st[1] != 1:
        raise ValueError(f"logits must be row-major, got stride {st}")
    return shape[0], shape[1], st[0] if shape[0] > 1 else shape[1], code


def bsmm_route_topk(logits, k, *, mask=None, renorm=True, alpha=None, workspace=None,
                    stream=None):
    """Top-k experts of every token, with what their products need.

    logits: bf16 or fp32 [T, E], unit stride along E.  mask: bool or uint8
    [T], false for tokens to leave out.  renorm: the weights of a token sum to
    one.  alpha: weight of the balance loss; None for serving (no loss).
    Returns a Route: index and weight [T, k], counts [E], offsets [E + 1] and
    order [T * k] (the slots t * k + j sorted by expert, for
    bsmm_w4_expert_mm), and with a loss live [1], prob_sum [E] and loss [1].
    workspace: None for a cached one, or a 16-byte aligned tensor of
    bsmm_route_workspace_bytes bytes.
    """
    T, E, ldl, code = _route_logits(logits)
    if not 1 <= k <= min(E, 32):
        raise ValueError(f"k must be 1 to 32 and at most E = {E}, got {k}")
    _, torch, _, _, i32, f32 = _DTYPES
    mp = None if mask is None else _route_mask(mask, T)
    _one_gpu("logits, mask and workspace", logits, mask,
             None if workspace is False else workspace)
    dev = logits.device
    # few allocations and views: a decode step is bound by the host
    S = T * k
    new = torch.empty_strided
    index = new((T, k), (k, 1), dtype=i32, device=dev)
    weight = new((T, k), (k, 1), dtype=f32, device=dev)
    ints = new((S + 2 * E + 2,), (1,), dtype=i32, device=dev)
    op = ints.data_ptr()
    cp = op + 4 * S
    hs = _stream(stream)
    lib = load()
    wsp, wsn = (_buffer(lib.bsmm_route_workspace_bytes(T, E), dev, stream, hs)
                if workspace is None else _given(workspace))
    lp = pp = tp = None
    if alpha is not None:
        sums = new((E + 1,), (1,), dtype=f32, device=dev)
        lp, pp = cp + 8 * E + 4, sums.data_ptr()
        tp = pp + 4 * E
    status = lib.bsmm_route_topk(
        logits.data_ptr(), ldl, code, mp, k, 1 if renorm else 0, alpha or 0.0, index.data_ptr(),
        weight.data_ptr(), cp, cp + 4 * E, op, lp, pp, tp, T, E, wsp, wsn, hs)
    if status:
        _check(status)
    order, counts, offsets, live = torch.unsafe_split_with_sizes(ints, (S, E, E + 1, 1))
    if alpha is None:
        return Route(index, weight, counts, offsets, order, None, None, None)
    prob_sum, total = torch.unsafe_split_with_sizes(sums, (E, 1))
    return Route(index, weight, counts, offsets, order, live, prob_sum, total)


def bsmm_route_topk_backward(logits, index, weight, counts, live, *, dweight=None, dloss=None,
                             alpha=0.0, mask=None, renorm=True, out=None, stream=None):
    """The logits' gradient of bsmm_route_topk.

    logits, mask, renorm and alpha as given to the forward call; index,
    weight, counts and live from its Route (counts and live may be sums over
    data-parallel ranks).  dweight: fp32 [T, k] or None; dloss: fp32 of one
    element or None.  Returns dlogits like logits.
    """
    T, E, ldl, code = _route_logits(logits)
    _, torch, dtypes, _, i32, f32 = _DTYPES
    if index.dim() != 2:
        raise ValueError("index must be 2-D [T, k]")
    shape = index.shape
    k = shape[1]
    if shape[0] != T or index.dtype is not i32 or not index.is_contiguous():
        raise ValueError(f"index must be contiguous int32 [{T}, k]")
    for t, n in ((weight, "weight"), (dweight, "dweight")):
        if t is not None and (t.dtype is not f32 or t.shape != shape or not t.is_contiguous()):
            raise ValueError(f"{n} must be contiguous fp32 [{T}, {k}]")
    cp = lp = None
    if dloss is not None:
        if dloss.dtype is not f32 or dloss.numel() != 1:
            raise ValueError("dloss must be one fp32 value")
        if counts is None or counts.dtype is not i32 or counts.shape != (E,) or \
                not counts.is_contiguous():
            raise ValueError(f"counts must be contiguous int32 [{E}]")
        if live is None or live.dtype is not i32 or live.numel() != 1:
            raise ValueError("live must be one int32 value")
        cp, lp = counts.data_ptr(), live.data_ptr()
    mp = None if mask is None else _route_mask(mask, T)
    _one_gpu("logits, index, weight, counts, live, dweight, dloss, mask and out", logits, index,
             weight if dweight is not None else None, counts if dloss is not None else None,
             live if dloss is not None else None, dweight, dloss, mask, out)
    o, ldd = _w4_out(out, T, E, code, torch, dtypes, logits.device)
    status = load().bsmm_route_topk_backward(
        logits.data_ptr(), ldl, code, mp, index.data_ptr(),
        None if weight is None else weight.data_ptr(), cp, lp, k, 1 if renorm else 0, alpha,
        None if dweight is None else dweight.data_ptr(),
        None if dloss is None else dloss.data_ptr(), o.data_ptr(), ldd, T, E, _stream(stream))
    if status:
        _check(status)
    return o


def bsmm_workspace_bytes(op, G, M, N, K, out_dtype):
    return load().bsmm_workspace_bytes(op, G, M, N, K, _dtype_code(out_dtype))


def bsmm_w4_workspace_bytes(x_dtype, E, R, S, N, K, group):
    """Workspace bytes bsmm_w4_expert_mm wants (bsmm_w4_mm: E = 1, R = S = M)."""
    return load().bsmm_w4_workspace_bytes(_float_code(x_dtype, "x_dtype"), E, R, S, N, K, group)


def bsmm_w4_plan_name(x_dtype, routed, E, R, S, N, K, group):
    """The kernel of a bsmm_w4_expert_mm (``routed``) or bsmm_w4_mm call: rows4,
    rows16, rows32, tile128 or tile256; None for sizes that have none."""
    name = load().bsmm_w4_plan_name(_float_code(x_dtype, "x_dtype"), 1 if routed else 0, E, R, S,
                                    N, K, group)
    return name and name.decode()


def bsmm_expert_mm_workspace_bytes(dtype, transposed, E, S, N, K):
    """Workspace bytes bsmm_expert_mm wants (transposed: w is contiguous along N)."""
    return load().bsmm_expert_mm_workspace_bytes(_float_code(dtype, "dtype"),
                                                 1 if transposed else 0, E, S, N, K)


def bsmm_expert_wgrad_workspace_bytes(dtype, checkpoint, E, Rx, S, N, K):
    """Workspace bytes bsmm_expert_wgrad wants for dy of ``dtype`` and x [Rx, K]."""
    return load().bsmm_expert_wgrad_workspace_bytes(_float_code(dtype, "dtype"),
                                                    1 if checkpoint else 0, E, Rx, S, N, K)


def bsmm_expert_mm_plan_name(dtype, transposed, E, S, N, K, *, aligned=True, workspace=None):
    """The kernel of a bsmm_expert_mm call and its ranges of K: (rows, wide128,
    wide192, wide256 or tile64, ranges); None for sizes that have none.
    aligned: whether rows are at multiples of 16 bytes.  workspace: its bytes,
    None for as many as the call wants."""
    code, parts = _float_code(dtype, "dtype"), ctypes.c_int(0)
    t = 1 if transposed else 0
    if workspace is None:
        workspace = load().bsmm_expert_mm_workspace_bytes(code, t, E, S, N, K)
    name = load().bsmm_expert_mm_plan_name(code, t, 1 if aligned else 0, E, S, N, K, workspace,
                                           ctypes.byref(parts))
    return name and (name.decode(), parts.value)


def bsmm_expert_wgrad_plan_name(dtype, checkpoint, E, Rx, S, N, K, *, out_dtype="f32",
                                dy_aligned=True, x_aligned=True, workspace=None):
    """The kernel of a bsmm_expert_wgrad call and its parts of the slots:
    (wide256, tile128, tile64 or restored, parts), as bsmm_expert_mm_plan_name.
    dy_aligned, x_aligned: whether row strides are multiples of 4 elements (a
    checkpoint's: rows at multiples of 8 bytes)."""
    code, parts = _float_code(dtype, "dtype"), ctypes.c_int(0)
    c = 1 if checkpoint else 0
    if workspace is None:
        workspace = load().bsmm_expert_wgrad_workspace_bytes(code, c, E, Rx, S, N, K)
    name = load().bsmm_expert_wgrad_plan_name(
        code, c, _float_code(out_dtype, "out_dtype"), 1 if dy_aligned else 0,
        1 if x_aligned else 0, E, Rx, S, N, K, workspace, ctypes.byref(parts))
    return name and (name.decode(), parts.value)


def bsmm_route_workspace_bytes(T, E):
    """Workspace bytes bsmm_route_topk needs."""
    return load().bsmm_route_workspace_bytes(T, E)


def bsmm_query_plan(op, G, M, N, K, out_dtype, workspace_bytes=2**62):
    info = PlanInfo()
    _check(load().bsmm_query_plan(op, G, M, N, K, _dtype_code(out_dtype),
                                  workspace_bytes, ctypes.byref(info)))
    return {"variant": info.variant.decode(), "tile_m": info.tile_m,
            "tile_n": info.tile_n, "split_k": info.split_k, "m_split": info.m_split,
            "workspace": info.workspace, "source": info.source,
            "tail_variant": info.tail_variant.decode(), "tail_split_k": info.tail_split_k}


def bsmm_set_override(variant=None, split_k=0):
    _WS_NEED.clear()              # the plans, and so their workspace, change
    _check(load().bsmm_set_override(variant.encode() if variant else None, split_k))


def bsmm_set_override_tail(m_split=0, tail_variant=None, tail_split=1):
    """Force an M-split (bulk rows [0, m_split), a tail launch of
    `tail_variant` with `tail_split` K slices) for the following calls;
    m_split 0 removes it (tests and tuning)."""
    _WS_NEED.clear()
    _check(load().bsmm_set_override_tail(int(m_split),
                                         tail_variant.encode() if tail_variant else None,
                                         int(tail_split)))


def bsmm_set_streamk_grid(workgroups=0):
    """Grid of the stream-K kernels for the following calls (0: as many
    workgroups as the device holds at once; tests and tuning)."""
    _WS_NEED.clear()
    _check(load().bsmm_set_streamk_grid(int(workgroups)))


def bsmm_mfma_probe(kind, workgroups, iters, out, stream=None):
    """Matrix-core throughput probe (kind 0: fp8 16x16x128, 1: int8
    16x16x64, 2: int8 32x32x32, 3: fp8 32x32x64); out: fp32 device tensor of
    workgroups * 256 elements.
    Returns the number of flops (ops) the launch performs."""
    if out.numel() < workgroups * 256:
        raise ValueError("out holds fewer than workgroups * 256 floats")
    _check(load().bsmm_mfma_probe(int(kind), int(workgroups), int(iters), out.data_ptr(),
                                  _stream(stream)))
    per = {0: 65536, 1: 32768, 2: 65536, 3: 131072}[kind]
    return float(workgroups) * 4 * iters * 8 * per


def bsmm_timing_enable(enable=True):
    """Time the main launch of every following call with HIP events."""
    _check(load().bsmm_timing_enable(1 if enable else 0))


def bsmm_timing_read():
    """(mean ms, launches, variant) of the launches timed since enabling."""
    ms, n = ctypes.c_double(), ctypes.c_int64()
    name = ctypes.create_string_buffer(64)
    _check(load().bsmm_timing_read(ctypes.byref(ms), ctypes.byref(n), name, 64))
    return ms.value, n.value, name.value.decode()


def bsmm_variant_names():
    return load().bsmm_variant_names().decode().split(",")


def bsmm_version():
    return load().bsmm_version()
