"""Python binding of the C ABI in ``include/moe_mxfp4.h`` (argument marshalling
only).  Every compute step runs in the library's CUDA kernels; torch supplies
device memory (tensors) and the current CUDA stream.  If the shared library is
missing the calls raise: there is no fallback path.
"""
from __future__ import annotations

import ctypes as C
import os
import threading

import torch

from . import build_lib

(MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_CUDA, MOE_ERR_DATA, MOE_ERR_TIMEOUT,
 MOE_ERR_CAPACITY) = range(7)
MOE_ROUTE_SORT_NOALLOC_SCRATCH_BYTES = 512 * 1024
MOE_F32, MOE_BF16 = 0, 1
MOE_ACT_ROW_MAJOR, MOE_ACT_K8_INTERLEAVED, MOE_ACT_K8_TOKEN_ORDER = 0, 1, 2
MOE_FP4_MX, MOE_FP4_NV = 0, 1

SYMBOLS = (
    "moe_status_string", "moe_workspace_bytes", "moe_clear_status", "moe_read_status",
    "moe_route_sort", "moe_mxfp4_grouped_gemm", "moe_swiglu", "moe_combine", "moe_layer_forward",
    "moe_mxfp4_decode_expert", "moe_debug_bounded_wait", "moe_last_launch_count",
    "moe_route_sort_noalloc", "moe_nvfp4_cast_workspace_bytes", "moe_mxfp4_to_nvfp4",
    "moe_nvfp4_grouped_gemm", "moe_mxfp4_grouped_gemm_swiglu", "moe_mxfp4_grouped_gemm_block",
    "moe_mxfp4_grouped_gemm_swiglu_gather", "moe_mxfp4_grouped_gemm_scatter", "moe_combine_slots",
    "moe_act_interleave_k8", "moe_set_gemm_pairing", "moe_topk_gate", "moe_topk_gate_backward",
    "moe_fp4_quantize", "moe_fp4_grouped_gemm", "moe_fp4_grouped_gemm_swiglu",
    "moe_layer_forward_fp4", "moe_combine_backward", "moe_gather_backward",
)

_lock = threading.Lock()
_lib = None


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


def library_path() -> str:
    return build_lib.LIB


def load(path: str | None = None):
    """Load the shared library (it must have been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            p = path or build_lib.LIB
            if not os.path.exists(p):
                raise RuntimeError(f"CUDA library not built: {p} (run __graft_entry__.build())")
            lib = C.CDLL(p)
            P, I32, I64, SZ, U64 = C.c_void_p, C.c_int32, C.c_int64, C.c_size_t, C.c_uint64
            sig = {
                "moe_status_string": ([C.c_int], C.c_char_p),
                "moe_workspace_bytes": ([I32, I32, I32], SZ),
                "moe_clear_status": ([P, P], C.c_int),
                "moe_read_status": ([P, P], C.c_int),
                "moe_route_sort": ([P, I32, I32, I32, P, P, P, P, P, I32, P, C.c_int, P, SZ, P], C.c_int),
                "moe_route_sort_noalloc": ([P, I32, I32, I32, P, P, P, P, P, I32, P, C.c_int, P],
                                           C.c_int),
                "moe_mxfp4_grouped_gemm": ([P, C.c_int, I64, I32, P, P, P, I32, I32, P, C.c_int, P, SZ,
                                            P], C.c_int),
                "moe_mxfp4_grouped_gemm_block": ([P, C.c_int, I64, I32, I32, P, P, P, I32, I32, P,
                                                  C.c_int, P, SZ, P], C.c_int),
                "moe_mxfp4_grouped_gemm_swiglu": ([P, C.c_int, I64, I32, P, P, P, I32, I32, P,
                                                   C.c_int, P, SZ, P], C.c_int),
                "moe_mxfp4_grouped_gemm_swiglu_gather": ([P, I32, I32, P, I64, I32, P, P, P, I32,
                                                          I32, P, C.c_int, P, SZ, P], C.c_int),
                "moe_mxfp4_grouped_gemm_scatter": ([P, C.c_int, I64, I32, P, P, P, I32, I32, P, P,
                                                    C.c_int, P, SZ, P], C.c_int),
                "moe_combine_slots": ([P, P, P, I32, I32, I32, P, C.c_int, P], C.c_int),
                "moe_act_interleave_k8": ([P, I64, I32, P, P], C.c_int),
                "moe_set_gemm_pairing": ([I32], C.c_int),
                "moe_swiglu": ([P, C.c_int, I64, I32, P, C.c_int, P], C.c_int),
                "moe_combine": ([P, P, P, I32, I32, I32, P, C.c_int, P], C.c_int),
                "moe_layer_forward": ([P, P, P, I32, I32, I32, I32, I32, P, P, P, P, P,
                                       P, P, P, P, P, P, P, P, SZ, P], C.c_int),
                "moe_mxfp4_decode_expert": ([P, P, I32, I32, I32, I32, P, P, SZ, P], C.c_int),
                "moe_debug_bounded_wait": ([U64, P, SZ, P], C.c_int),
                "moe_last_launch_count": ([], I32),
                "moe_nvfp4_cast_workspace_bytes": ([I32], SZ),
                "moe_mxfp4_to_nvfp4": ([P, I32, I32, I32, P, P, P, P, SZ, P], C.c_int),
                "moe_nvfp4_grouped_gemm": ([P, C.c_int, I64, I32, P, P, P, P, I32, I32, P, C.c_int,
                                            P, SZ, P], C.c_int),
                "moe_topk_gate": ([P, C.c_int, I64, I32, I32, I32, I32, P, P, P], C.c_int),
                "moe_topk_gate_backward": ([P, C.c_int, I64, I32, I32, I32, I32, P, P, P, P], C.c_int),
                "moe_fp4_quantize": ([P, C.c_int, I64, I64, I32, P, I32, I64, C.c_int, P, P, P, P,
                                      C.c_int, P, SZ, P], C.c_int),
                "moe_fp4_grouped_gemm": ([P, P, P, I64, I32, P, P, P, C.c_int, P, I32, I32, P, C.c_int,
                                          P, SZ, P], C.c_int),
                "moe_fp4_grouped_gemm_swiglu": ([P, P, P, I64, I32, P, P, P, C.c_int, P, I32, I32, P, P,
                                                 P, P, SZ, P], C.c_int),
                "moe_layer_forward_fp4": ([P, P, P, I32, I32, I32, I32, I32, C.c_int] + [P] * 18 +
                                          [P, SZ, P], C.c_int),
                "moe_combine_backward": ([P, C.c_int, P, C.c_int, P, P, I32, I32, I32, P, C.c_int, P, P],
                                         C.c_int),
                "moe_gather_backward": ([P, C.c_int, P, I32, I32, I32, P, C.c_int, P], C.c_int),
            }
            for name, (args, res) in sig.items():
                f = getattr(lib, name)
                f.argtypes = args
                f.restype = res
            _lib = lib
    return _lib


def status_string(status: int) -> str:
    try:
        return load().moe_status_string(int(status)).decode()
    except RuntimeError:
        return f"status {status}"


def _ptr(t):
    return None if t is None else t.data_ptr()


# The current stream's handle without building a Stream object (4 us a call, as
# long as a small kernel), where torch has the calls for it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream=None):
    if stream is None and _raw_stream and _raw_device and torch.cuda.is_initialized():
        return _raw_stream(_raw_device())
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _empty(shape, dtype, device, stream):
    """torch.empty of the pool of the stream that the call runs on: given back, the memory
    then goes to work that comes after the call's."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):       # anything with the handle, as _stream takes it
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _check(rc: int, where: str):
    if rc != MOE_OK:
        raise MoeError(rc, where)


def _dtype_code(dt) -> int:
    if dt == torch.float32:
        return MOE_F32
    if dt == torch.bfloat16:
        return MOE_BF16
    raise ValueError(f"unsupported dtype {dt}")


MOE_PAIRING_AUTO, MOE_PAIRING_OFF, MOE_PAIRING_ON = 0, 1, 2


def set_gemm_pairing(mode: int):
    """CTA pairs for bands over 32 rows: MOE_PAIRING_AUTO / _OFF / _ON (process-wide)."""
    _check(load().moe_set_gemm_pairing(int(mode)), "moe_set_gemm_pairing")


def last_launch_count() -> int:
    return int(load().moe_last_launch_count())


# ---------------------------------------------------------------- workspace

def workspace_bytes(T: int, k: int, E: int) -> int:
    return int(load().moe_workspace_bytes(T, k, E))


def make_workspace(T: int, k: int, E: int, device="cuda", stream=None) -> torch.Tensor:
    ws = _empty(workspace_bytes(T, k, E), torch.uint8, device, stream)
    clear_status(ws, stream)
    return ws


def clear_status(workspace: torch.Tensor, stream=None):
    _check(load().moe_clear_status(_ptr(workspace), _stream(stream)), "moe_clear_status")


def read_status(workspace: torch.Tensor, stream=None) -> int:
    return int(load().moe_read_status(_ptr(workspace), _stream(stream)))


# ---------------------------------------------------------------- operations

def route_sort(topk_ids: torch.Tensor, E: int, x: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None, out=None, stream=None,
               x_layout: int = MOE_ACT_ROW_MAJOR):
    """Returns (group_sizes[E], group_offsets[E+1], sorted_slot[T*k],
    slot_to_row[T*k], x_sorted or None); x_sorted in `x_layout` order
    (MOE_ACT_K8_TOKEN_ORDER: x itself [T, hidden] in the K8 order)."""
    T, k = topk_ids.shape
    dev = topk_ids.device
    rows = T * k
    if out is None:
        gs = torch.empty(E, dtype=torch.int32, device=dev)
        off = torch.empty(E + 1, dtype=torch.int32, device=dev)
        ss = torch.empty(rows, dtype=torch.int32, device=dev)
        s2r = torch.empty(rows, dtype=torch.int32, device=dev)
        xs_rows = T if x_layout == MOE_ACT_K8_TOKEN_ORDER else rows
        xs = None if x is None else torch.empty((xs_rows, x.shape[1]), dtype=x.dtype, device=dev)
    else:
        gs, off, ss, s2r, xs = out
    if workspace is None:
        workspace = make_workspace(T, k, E, dev, stream)
    hidden = 0 if x is None else x.shape[1]
    rc = load().moe_route_sort(_ptr(topk_ids), T, k, E, _ptr(gs), _ptr(off), _ptr(ss), _ptr(s2r),
                               _ptr(x), hidden, _ptr(xs), x_layout, _ptr(workspace),
                               workspace.numel(), _stream(stream))
    _check(rc, "moe_route_sort")
    return gs, off, ss, s2r, xs


def route_sort_noalloc(topk_ids: torch.Tensor, E: int, out, x: torch.Tensor | None = None,
                       stream=None, x_layout: int = MOE_ACT_ROW_MAJOR):
    """Route sort through the fixed-capacity entry point, for callers that must
    not allocate at the point of the call.  `out` = (group_sizes, group_offsets,
    sorted_slot, slot_to_row, x_sorted or None) must already exist: this wrapper
    creates no tensor, and the library call uses its own static scratch instead
    of a workspace.  Raises MoeError(MOE_ERR_CAPACITY) when the problem needs
    more than MOE_ROUTE_SORT_NOALLOC_SCRATCH_BYTES of scratch."""
    T, k = topk_ids.shape
    gs, off, ss, s2r, xs = out
    hidden = 0 if x is None else x.shape[1]
    rc = load().moe_route_sort_noalloc(_ptr(topk_ids), T, k, E, _ptr(gs), _ptr(off), _ptr(ss),
                                       _ptr(s2r), _ptr(x), hidden, _ptr(xs), x_layout,
                                       _stream(stream))
    _check(rc, "moe_route_sort_noalloc")
    return out


def grouped_gemm(act: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                 group_sizes: torch.Tensor, out: torch.Tensor | None = None,
                 out_dtype=torch.float32, workspace: torch.Tensor | None = None, stream=None,
                 act_layout: int = MOE_ACT_ROW_MAJOR):
    """act bf16 [rows, K] (row-major or K8-interleaved); codes uint8 [E, N, K/2];
    scales uint8 [E, N, K/32]; group_sizes int32 [E] -> out [rows, N] (f32 or bf16)."""
    rows, K = act.shape
    E, N, _ = codes.shape
    if out is None:
        out = torch.empty((rows, N), dtype=out_dtype, device=act.device)
    if workspace is None:
        workspace = make_workspace(0, 1, 1, act.device, stream)
    rc = load().moe_mxfp4_grouped_gemm(_ptr(act), act_layout, rows, K, _ptr(codes), _ptr(scales),
                                       _ptr(group_sizes), E, N, _ptr(out), _dtype_code(out.dtype),
                                       _ptr(workspace), workspace.numel(), _stream(stream))
    _check(rc, "moe_mxfp4_grouped_gemm")
    return out


def grouped_gemm_block(act: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                       group_sizes: torch.Tensor, scale_block: int, out: torch.Tensor | None = None,
                       out_dtype=torch.float32, workspace: torch.Tensor | None = None, stream=None,
                       act_layout: int = MOE_ACT_ROW_MAJOR):
    """grouped_gemm with one E8M0 scale per `scale_block` (32 or 512)
    consecutive k: scales uint8 [E, N, K / scale_block]."""
    rows, K = act.shape
    E, N, _ = codes.shape
    if out is None:
        out = torch.empty((rows, N), dtype=out_dtype, device=act.device)
    if workspace is None:
        workspace = make_workspace(0, 1, 1, act.device, stream)
    rc = load().moe_mxfp4_grouped_gemm_block(_ptr(act), act_layout, rows, K, int(scale_block),
                                             _ptr(codes), _ptr(scales), _ptr(group_sizes), E, N,
                                             _ptr(out), _dtype_code(out.dtype), _ptr(workspace),
                                             workspace.numel(), _stream(stream))
    _check(rc, "moe_mxfp4_grouped_gemm_block")
    return out


def grouped_gemm_swiglu(act: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                        group_sizes: torch.Tensor, out: torch.Tensor | None = None,
                        workspace: torch.Tensor | None = None, stream=None,
                        act_layout: int = MOE_ACT_ROW_MAJOR, h_layout: int = MOE_ACT_ROW_MAJOR):
    """w13 grouped GEMM with SwiGLU in its epilogue.  act bf16 [rows, K]; codes
    uint8 [E, 2I, K/2] and scales uint8 [E, 2I, K/32] with gate rows [0, I) and
    up rows [I, 2I); group_sizes int32 [E] -> h bf16 [rows, I] in `h_layout`."""
    rows, K = act.shape
    E, two_i, _ = codes.shape
    I = two_i // 2
    if out is None:
        out = torch.empty((rows, I), dtype=torch.bfloat16, device=act.device)
    if workspace is None:
        workspace = make_workspace(0, 1, 1, act.device, stream)
    rc = load().moe_mxfp4_grouped_gemm_swiglu(_ptr(act), act_layout, rows, K, _ptr(codes),
                                              _ptr(scales), _ptr(group_sizes), E, I, _ptr(out),
                                              h_layout, _ptr(workspace), workspace.numel(),
                                              _stream(stream))
    _check(rc, "moe_mxfp4_grouped_gemm_swiglu")
    return out


def grouped_gemm_swiglu_gather(x_k8: torch.Tensor, top_k: int, sorted_slot: torch.Tensor,
                               codes: torch.Tensor, scales: torch.Tensor,
                               group_sizes: torch.Tensor, out: torch.Tensor | None = None,
                               workspace: torch.Tensor | None = None, stream=None,
                               h_layout: int = MOE_ACT_ROW_MAJOR):
    """grouped_gemm_swiglu with the activation rows gathered in the load: sorted
    row r reads row sorted_slot[r] // top_k of x_k8 bf16 [T, K] (K8-interleaved);
    -> h bf16 [rows, I], rows = sorted_slot.numel()."""
    T, K = x_k8.shape
    rows = sorted_slot.numel()
    E, two_i, _ = codes.shape
    I = two_i // 2
    if out is None:
        out = torch.empty((rows, I), dtype=torch.bfloat16, device=x_k8.device)
    if workspace is None:
        workspace = make_workspace(0, 1, 1, x_k8.device, stream)
    rc = load().moe_mxfp4_grouped_gemm_swiglu_gather(
        _ptr(x_k8), T, int(top_k), _ptr(sorted_slot), rows, K, _ptr(codes), _ptr(scales),
        _ptr(group_sizes), E, I, _ptr(out), h_layout, _ptr(workspace), workspace.numel(),
        _stream(stream))
    _check(rc, "moe_mxfp4_grouped_gemm_swiglu_gather")
    return out


def grouped_gemm_scatter(act: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                         group_sizes: torch.Tensor, out_row: torch.Tensor,
                         out: torch.Tensor | None = None, out_dtype=torch.float32,
                         workspace: torch.Tensor | None = None, stream=None,
                         act_layout: int = MOE_ACT_ROW_MAJOR):
    """grouped_gemm writing sorted row r to row out_row[r] of out [rows, N]."""
    rows, K = act.shape
    E, N, _ = codes.shape
    if out is None:
        out = torch.empty((rows, N), dtype=out_dtype, device=act.device)
    if workspace is None:
        workspace = make_workspace(0, 1, 1, act.device, stream)
    rc = load().moe_mxfp4_grouped_gemm_scatter(_ptr(act), act_layout, rows, K, _ptr(codes),
                                               _ptr(scales), _ptr(group_sizes), E, N,
                                               _ptr(out_row), _ptr(out), _dtype_code(out.dtype),
                                               _ptr(workspace), workspace.numel(), _stream(stream))
    _check(rc, "moe_mxfp4_grouped_gemm_scatter")
    return out


def act_interleave_k8(x: torch.Tensor, out: torch.Tensor | None = None, stream=None):
    """bf16 [rows, hidden] -> the same rows in the K8-interleaved order."""
    rows, hidden = x.shape
    if out is None:
        out = torch.empty_like(x)
    rc = load().moe_act_interleave_k8(_ptr(x), rows, hidden, _ptr(out), _stream(stream))
    _check(rc, "moe_act_interleave_k8")
    return out


def nvfp4_grouped_gemm(act: torch.Tensor, codes: torch.Tensor, scales16: torch.Tensor,
                       weight_scale_2: torch.Tensor, group_sizes: torch.Tensor,
                       out: torch.Tensor | None = None, out_dtype=torch.float32,
                       workspace: torch.Tensor | None = None, stream=None,
                       act_layout: int = MOE_ACT_ROW_MAJOR):
    """act bf16 [rows, K]; codes uint8 [E, N, K/2]; scales16 uint8 [E, N, K/16]
    (E4M3); weight_scale_2 f32 [E]; group_sizes int32 [E] -> out [rows, N]."""
    rows, K = act.shape
    E, N, _ = codes.shape
    if out is None:
        out = torch.empty((rows, N), dtype=out_dtype, device=act.device)
    if workspace is None:
        workspace = make_workspace(0, 1, 1, act.device, stream)
    rc = load().moe_nvfp4_grouped_gemm(_ptr(act), act_layout, rows, K, _ptr(codes), _ptr(scales16),
                                       _ptr(weight_scale_2), _ptr(group_sizes), E, N, _ptr(out),
                                       _dtype_code(out.dtype), _ptr(workspace), workspace.numel(),
                                       _stream(stream))
    _check(rc, "moe_nvfp4_grouped_gemm")
    return out


def swiglu(gu: torch.Tensor, out: torch.Tensor | None = None, stream=None,
           layout: int = MOE_ACT_ROW_MAJOR):
    rows, two_i = gu.shape
    I = two_i // 2
    if out is None:
        out = torch.empty((rows, I), dtype=torch.bfloat16, device=gu.device)
    rc = load().moe_swiglu(_ptr(gu), _dtype_code(gu.dtype), rows, I, _ptr(out), layout,
                           _stream(stream))
    _check(rc, "moe_swiglu")
    return out


def combine(y: torch.Tensor, slot_to_row: torch.Tensor, topk_w: torch.Tensor,
            out: torch.Tensor | None = None, out_dtype=torch.float32, stream=None):
    T, k = topk_w.shape
    N = y.shape[1]
    if out is None:
        out = torch.empty((T, N), dtype=out_dtype, device=y.device)
    rc = load().moe_combine(_ptr(y), _ptr(slot_to_row), _ptr(topk_w), T, k, N, _ptr(out),
                            _dtype_code(out.dtype), _stream(stream))
    _check(rc, "moe_combine")
    return out


def combine_slots(y: torch.Tensor, slot_to_row: torch.Tensor, topk_w: torch.Tensor,
                  out: torch.Tensor | None = None, out_dtype=torch.float32, stream=None):
    """combine with y f32 [T*k, N] in slot order (slot_to_row marks valid slots)."""
    T, k = topk_w.shape
    N = y.shape[1]
    if out is None:
        out = torch.empty((T, N), dtype=out_dtype, device=y.device)
    rc = load().moe_combine_slots(_ptr(y), _ptr(slot_to_row), _ptr(topk_w), T, k, N, _ptr(out),
                                  _dtype_code(out.dtype), _stream(stream))
    _check(rc, "moe_combine_slots")
    return out


class LayerBuffers:
    """Caller-owned intermediates of one layer pass (allocated once, reused)."""

    def __init__(self, T: int, k: int, E: int, hidden: int, inter: int, device="cuda"):
        rows = T * k
        i32 = dict(dtype=torch.int32, device=device)
        self.group_sizes = torch.empty(E, **i32)
        self.group_offsets = torch.empty(E + 1, **i32)
        self.sorted_slot = torch.empty(rows, **i32)
        self.slot_to_row = torch.empty(rows, **i32)
        self.x_sorted = torch.empty((rows, hidden), dtype=torch.bfloat16, device=device)
        self.h = torch.empty((rows, inter), dtype=torch.bfloat16, device=device)
        self.y2 = torch.empty((rows, hidden), dtype=torch.float32, device=device)
        self.out = torch.empty((T, hidden), dtype=torch.float32, device=device)
        self.workspace = make_workspace(T, k, E, device)


def layer_forward(x, topk_ids, topk_w, w13_codes, w13_scales, w2_codes, w2_scales,
                  buffers: LayerBuffers, stream=None):
    T, k = topk_ids.shape
    E, two_i, hidden_half = w13_codes.shape
    hidden, inter = 2 * hidden_half, two_i // 2
    b = buffers
    rc = load().moe_layer_forward(
        _ptr(x), _ptr(topk_ids), _ptr(topk_w), T, k, E, hidden, inter,
        _ptr(w13_codes), _ptr(w13_scales), _ptr(w2_codes), _ptr(w2_scales), _ptr(b.out),
        _ptr(b.group_sizes), _ptr(b.group_offsets), _ptr(b.sorted_slot), _ptr(b.slot_to_row),
        _ptr(b.x_sorted), _ptr(b.h), _ptr(b.y2), _ptr(b.workspace),
        b.workspace.numel(), _stream(stream))
    _check(rc, "moe_layer_forward")
    return b.out


def decode_expert(codes: torch.Tensor, scales: torch.Tensor, e: int,
                  workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    E, N, Kh = codes.shape
    K = 2 * Kh
    out = torch.empty((N, K), dtype=torch.bfloat16, device=codes.device)
    if workspace is None:
        workspace = make_workspace(0, 1, 1, codes.device, stream)
    rc = load().moe_mxfp4_decode_expert(_ptr(codes), _ptr(scales), E, N, K, e, _ptr(out),
                                        _ptr(workspace), workspace.numel(), _stream(stream))
    _check(rc, "moe_mxfp4_decode_expert")
    return out


def mxfp4_to_nvfp4(scales: torch.Tensor, out=None, workspace: torch.Tensor | None = None,
                   stream=None):
    """Lossless MXFP4 -> NVFP4 scale cast.  scales uint8 [E, N, K/32] ->
    (e4m3 uint8 [E, N, K/16], weight_scale_2 f32 [E], out_of_range int64 [E]);
    `out` may hold those three tensors already (out_of_range holds the uint64
    counts of the C call, which never exceed 2^63)."""
    E, N, Kb = scales.shape
    dev = scales.device
    if out is None:
        out = (torch.empty((E, N, 2 * Kb), dtype=torch.uint8, device=dev),
               torch.empty(E, dtype=torch.float32, device=dev),
               torch.empty(E, dtype=torch.int64, device=dev))
    e4m3, ws2, oob = out
    if workspace is None:
        workspace = _empty(int(load().moe_nvfp4_cast_workspace_bytes(E)), torch.uint8, dev, stream)
        clear_status(workspace, stream)
    rc = load().moe_mxfp4_to_nvfp4(_ptr(scales), E, N, 32 * Kb, _ptr(e4m3), _ptr(ws2), _ptr(oob),
                                   _ptr(workspace), workspace.numel(), _stream(stream))
    _check(rc, "moe_mxfp4_to_nvfp4")
    return out


# ------------------------------------------- router gate, 4-bit path, gradients

def _need(name: str, t: torch.Tensor, shape, *dtypes):
    """The library takes raw pointers: a tensor it would misread is refused here."""
    if t.dtype in dtypes and t.shape == shape and t.is_contiguous() and t.is_cuda:
        return
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: not contiguous")
    raise ValueError(f"{name}: not a CUDA tensor")


def _room(name: str, t: torch.Tensor, n: int, dtype):
    """A buffer with room for n elements, which the call lays out itself."""
    if not (t.numel() >= n and t.dtype == dtype and t.is_contiguous() and t.is_cuda):
        raise ValueError(f"{name}: {t.numel()} elements of {t.dtype}, {n} of {dtype} in contiguous CUDA memory are needed")


def _workspace(ws, device, stream):
    """The call's workspace: the caller's, if the kernels can write it, or a new one."""
    if ws is None:
        return make_workspace(0, 1, 1, device, stream)
    if not (ws.is_cuda and ws.is_contiguous()):
        raise ValueError("workspace: a contiguous CUDA tensor is needed")
    return ws


def _rows_of(name: str, t: torch.Tensor) -> int:
    """Row stride, in elements, of a 2-D tensor whose rows are contiguous."""
    if t.dim() != 2 or t.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"{name}: a 2-D float32 or bfloat16 tensor is needed")
    if not t.is_cuda:
        raise ValueError(f"{name}: not a CUDA tensor")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: rows are not contiguous")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def topk_gate(logits: torch.Tensor, k: int, renorm: bool = False, out=None, stream=None):
    """Router gate: logits [T, E] (f32 or bf16, any row stride) -> (ids int32 [T, k],
    weights f32 [T, k]): the k largest, ties to the lower expert, and softmax over all
    E (renorm: over the chosen k) at them."""
    stride = _rows_of("logits", logits)
    T, E = logits.shape
    if out is None:
        out = (_empty((T, k), torch.int32, logits.device, stream),
               _empty((T, k), torch.float32, logits.device, stream))
    ids, w = out
    _need("ids", ids, (T, k), torch.int32)
    _need("weights", w, (T, k), torch.float32)
    rc = load().moe_topk_gate(_ptr(logits), _dtype_code(logits.dtype), stride, T, E, int(k),
                              int(bool(renorm)), _ptr(ids), _ptr(w), _stream(stream))
    _check(rc, "moe_topk_gate")
    return out


def topk_gate_backward(logits: torch.Tensor, ids: torch.Tensor, dw: torch.Tensor, renorm: bool = False,
                       out: torch.Tensor | None = None, stream=None):
    """Gradient of topk_gate's weights: dw f32 [T, k] -> dlogits [T, E] of the logits' type."""
    stride = _rows_of("logits", logits)
    T, E = logits.shape
    k = ids.shape[1] if ids.dim() == 2 else 0
    _need("ids", ids, (T, k), torch.int32)
    _need("dw", dw, (T, k), torch.float32)
    if out is None:
        out = _empty((T, E), logits.dtype, logits.device, stream)
    _need("dlogits", out, (T, E), logits.dtype)
    rc = load().moe_topk_gate_backward(_ptr(logits), _dtype_code(logits.dtype), stride, T, E, k,
                                       int(bool(renorm)), _ptr(ids), _ptr(dw), _ptr(out), _stream(stream))
    _check(rc, "moe_topk_gate_backward")
    return out


def _fp4_block(fmt: int) -> int:
    if fmt not in (MOE_FP4_MX, MOE_FP4_NV):
        raise ValueError(f"unknown 4-bit format {fmt}")
    return 32 if fmt == MOE_FP4_MX else 16


def _tensor_scale(name: str, t, n: int, fmt: int):
    if fmt == MOE_FP4_NV:
        if t is None:
            raise ValueError(f"{name} is needed for NVFP4")
        _need(name, t, (n,), torch.float32)
        return _ptr(t)
    return None


def fp4_quantize(x: torch.Tensor, fmt: int, row_index: torch.Tensor | None = None, index_div: int = 1,
                 tensor_scale: torch.Tensor | None = None, out=None, values: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, stream=None):
    """x [x_rows, K] (f32 or bf16, any row stride) -> (codes uint8 [rows, K/2], scales uint8
    [rows, K/32 or K/16]).  With row_index int32 [rows] row r holds x[row_index[r] // index_div].
    tensor_scale f32 [1] (NVFP4).  values (f32 or bf16 [rows, K]) receives what the codes
    stand for.  Bad indices and tensor scales are reported in the workspace (read_status):
    without one the call makes its own, whose status nobody sees."""
    stride = _rows_of("x", x)
    block = _fp4_block(fmt)
    x_rows, K = x.shape
    rows = x_rows if row_index is None else row_index.numel()
    if row_index is not None:
        _need("row_index", row_index, (rows,), torch.int32)
    if out is None:
        out = (_empty((rows, K // 2), torch.uint8, x.device, stream),
               _empty((rows, K // block), torch.uint8, x.device, stream))
    codes, scales = out
    _need("codes", codes, (rows, K // 2), torch.uint8)
    _need("scales", scales, (rows, K // block), torch.uint8)
    vdt = MOE_F32
    if values is not None:
        _need("values", values, (rows, K), torch.float32, torch.bfloat16)
        vdt = _dtype_code(values.dtype)
    workspace = _workspace(workspace, x.device, stream)
    rc = load().moe_fp4_quantize(_ptr(x), _dtype_code(x.dtype), x_rows, stride, K, _ptr(row_index),
                                 int(index_div), rows, fmt,
                                 _tensor_scale("tensor_scale", tensor_scale, 1, fmt), _ptr(codes),
                                 _ptr(scales), _ptr(values), vdt, _ptr(workspace), workspace.numel(),
                                 _stream(stream))
    _check(rc, "moe_fp4_quantize")
    return out


def _fp4_operands(act_codes, act_scales, codes, scales, group_sizes, fmt):
    block = _fp4_block(fmt)
    rows, half = act_codes.shape
    E, N, _ = codes.shape
    K = 2 * half
    _need("act_codes", act_codes, (rows, half), torch.uint8)
    _need("act_scales", act_scales, (rows, K // block), torch.uint8)
    _need("codes", codes, (E, N, half), torch.uint8)
    _need("scales", scales, (E, N, K // block), torch.uint8)
    _need("group_sizes", group_sizes, (E,), torch.int32)
    return rows, K, E, N, block


def fp4_grouped_gemm(act_codes: torch.Tensor, act_scales: torch.Tensor, codes: torch.Tensor,
                     scales: torch.Tensor, group_sizes: torch.Tensor, fmt: int,
                     act_scale_2: torch.Tensor | None = None,
                     weight_scale_2: torch.Tensor | None = None, out: torch.Tensor | None = None,
                     out_dtype=torch.float32, workspace: torch.Tensor | None = None, stream=None):
    """4-bit activations (fp4_quantize) by 4-bit weights uint8 [E, N, K/2] with scales
    [E, N, K/32 or K/16] over row bands group_sizes int32 [E] -> out [rows, N] (f32 or bf16).
    NVFP4: act_scale_2 f32 [1] and weight_scale_2 f32 [E].  Bad scales and group sizes are
    reported in the workspace (read_status), as for fp4_quantize."""
    rows, K, E, N, _ = _fp4_operands(act_codes, act_scales, codes, scales, group_sizes, fmt)
    if out is None:
        out = _empty((rows, N), out_dtype, act_codes.device, stream)
    _need("out", out, (rows, N), torch.float32, torch.bfloat16)
    workspace = _workspace(workspace, act_codes.device, stream)
    rc = load().moe_fp4_grouped_gemm(_ptr(act_codes), _ptr(act_scales),
                                     _tensor_scale("act_scale_2", act_scale_2, 1, fmt), rows, K,
                                     _ptr(codes), _ptr(scales),
                                     _tensor_scale("weight_scale_2", weight_scale_2, E, fmt), fmt,
                                     _ptr(group_sizes), E, N, _ptr(out), _dtype_code(out.dtype),
                                     _ptr(workspace), workspace.numel(), _stream(stream))
    _check(rc, "moe_fp4_grouped_gemm")
    return out


def fp4_grouped_gemm_swiglu(act_codes: torch.Tensor, act_scales: torch.Tensor, codes: torch.Tensor,
                            scales: torch.Tensor, group_sizes: torch.Tensor, fmt: int,
                            act_scale_2: torch.Tensor | None = None,
                            weight_scale_2: torch.Tensor | None = None,
                            h_scale_2: torch.Tensor | None = None, out=None,
                            workspace: torch.Tensor | None = None, stream=None):
    """The w13 product (codes [E, 2I, K/2], gate rows first) with SwiGLU and the
    quantisation of h in its epilogue -> (h_codes uint8 [rows, I/2], h_scales uint8
    [rows, I/32 or I/16]).  Workspace as for fp4_grouped_gemm."""
    rows, K, E, N, block = _fp4_operands(act_codes, act_scales, codes, scales, group_sizes, fmt)
    if N % 2:
        raise ValueError("codes: an odd number of gate and up rows")
    I = N // 2
    if out is None:
        out = (_empty((rows, I // 2), torch.uint8, act_codes.device, stream),
               _empty((rows, I // block), torch.uint8, act_codes.device, stream))
    h_codes, h_scales = out
    _need("h_codes", h_codes, (rows, I // 2), torch.uint8)
    _need("h_scales", h_scales, (rows, I // block), torch.uint8)
    workspace = _workspace(workspace, act_codes.device, stream)
    rc = load().moe_fp4_grouped_gemm_swiglu(
        _ptr(act_codes), _ptr(act_scales), _tensor_scale("act_scale_2", act_scale_2, 1, fmt), rows, K,
        _ptr(codes), _ptr(scales), _tensor_scale("weight_scale_2", weight_scale_2, E, fmt), fmt,
        _ptr(group_sizes), E, I, _tensor_scale("h_scale_2", h_scale_2, 1, fmt), _ptr(h_codes),
        _ptr(h_scales), _ptr(workspace), workspace.numel(), _stream(stream))
    _check(rc, "moe_fp4_grouped_gemm_swiglu")
    return out


def combine_backward(dout: torch.Tensor, y: torch.Tensor, slot_to_row: torch.Tensor,
                     topk_w: torch.Tensor, out=None, dy_dtype=None, stream=None):
    """Gradient of combine: dout [T, N], y [T*k, N] (f32 or bf16 each) -> (dy [T*k, N] of
    dy_dtype (default: dout's), dw f32 [T, k])."""
    T, k = topk_w.shape
    N = dout.shape[-1]
    _need("dout", dout, (T, N), torch.float32, torch.bfloat16)
    _need("y", y, (T * k, N), torch.float32, torch.bfloat16)
    _need("slot_to_row", slot_to_row, (T * k,), torch.int32)
    _need("topk_w", topk_w, (T, k), torch.float32)
    if out is None:
        out = (_empty((T * k, N), dy_dtype or dout.dtype, dout.device, stream),
               _empty((T, k), torch.float32, dout.device, stream))
    dy, dw = out
    _need("dy", dy, (T * k, N), torch.float32, torch.bfloat16)
    _need("dw", dw, (T, k), torch.float32)
    rc = load().moe_combine_backward(_ptr(dout), _dtype_code(dout.dtype), _ptr(y), _dtype_code(y.dtype),
                                     _ptr(slot_to_row), _ptr(topk_w), T, k, N, _ptr(dy),
                                     _dtype_code(dy.dtype), _ptr(dw), _stream(stream))
    _check(rc, "moe_combine_backward")
    return out


def gather_backward(dx_sorted: torch.Tensor, slot_to_row: torch.Tensor, k: int,
                    out: torch.Tensor | None = None, stream=None):
    """Gradient of route_sort's gather: dx_sorted [T*k, hidden] (f32 or bf16) -> dx [T, hidden]."""
    rows, hidden = dx_sorted.shape
    if k < 1 or rows % k:
        raise ValueError("dx_sorted: rows are not a multiple of k")
    T = rows // k
    _need("dx_sorted", dx_sorted, (rows, hidden), torch.float32, torch.bfloat16)
    _need("slot_to_row", slot_to_row, (rows,), torch.int32)
    if out is None:
        out = _empty((T, hidden), dx_sorted.dtype, dx_sorted.device, stream)
    _need("dx", out, (T, hidden), torch.float32, torch.bfloat16)
    rc = load().moe_gather_backward(_ptr(dx_sorted), _dtype_code(dx_sorted.dtype), _ptr(slot_to_row), T,
                                    int(k), hidden, _ptr(out), _dtype_code(out.dtype), _stream(stream))
    _check(rc, "moe_gather_backward")
    return out


class LayerBuffersFp4:
    """Caller-owned intermediates of one 4-bit layer pass (allocated once, reused by every
    call of at most T tokens and T * k rows)."""

    def __init__(self, T: int, k: int, E: int, hidden: int, inter: int, fmt: int, device="cuda"):
        rows, block = T * k, _fp4_block(fmt)
        i32 = dict(dtype=torch.int32, device=device)
        u8 = dict(dtype=torch.uint8, device=device)
        self.fmt = fmt
        self.group_sizes = torch.empty(E, **i32)
        self.group_offsets = torch.empty(E + 1, **i32)
        self.sorted_slot = torch.empty(rows, **i32)
        self.slot_to_row = torch.empty(rows, **i32)
        self.x_codes = torch.empty((rows, hidden // 2), **u8)
        self.x_scales = torch.empty((rows, hidden // block), **u8)
        self.h_codes = torch.empty((rows, inter // 2), **u8)
        self.h_scales = torch.empty((rows, inter // block), **u8)
        self.y2 = torch.empty((rows, hidden), dtype=torch.float32, device=device)
        self.out = torch.empty((T, hidden), dtype=torch.float32, device=device)
        self.workspace = make_workspace(T, k, E, device)


def layer_forward_fp4(x, topk_ids, topk_w, w13, w2, buffers: LayerBuffersFp4, x_scale_2=None,
                      h_scale_2=None, stream=None):
    """The routed-expert layer with 4-bit activations and weights.  w13 and w2 are (codes,
    scales, weight_scale_2 or None); x bf16 [T, hidden]; -> the first T rows of buffers.out, f32
    [T, hidden]."""
    b, fmt = buffers, buffers.fmt
    block = _fp4_block(fmt)
    (c13, s13, g13), (c2, s2, g2) = w13, w2
    T, k = topk_ids.shape
    E, two_i, half = c13.shape
    hidden, inter = 2 * half, two_i // 2
    _need("x", x, (T, hidden), torch.bfloat16)
    _need("topk_ids", topk_ids, (T, k), torch.int32)
    _need("topk_w", topk_w, (T, k), torch.float32)
    _need("w13 codes", c13, (E, 2 * inter, hidden // 2), torch.uint8)
    _need("w13 scales", s13, (E, 2 * inter, hidden // block), torch.uint8)
    _need("w2 codes", c2, (E, hidden, inter // 2), torch.uint8)
    _need("w2 scales", s2, (E, hidden, inter // block), torch.uint8)
    rows = T * k
    _room("buffers.x_codes", b.x_codes, rows * hidden // 2, torch.uint8)
    _room("buffers.x_scales", b.x_scales, rows * hidden // block, torch.uint8)
    _room("buffers.h_codes", b.h_codes, rows * inter // 2, torch.uint8)
    _room("buffers.h_scales", b.h_scales, rows * inter // block, torch.uint8)
    _room("buffers.y2", b.y2, rows * hidden, torch.float32)
    _room("buffers.out", b.out, T * hidden, torch.float32)
    _room("buffers.group_sizes", b.group_sizes, E, torch.int32)
    _room("buffers.group_offsets", b.group_offsets, E + 1, torch.int32)
    _room("buffers.sorted_slot", b.sorted_slot, rows, torch.int32)
    _room("buffers.slot_to_row", b.slot_to_row, rows, torch.int32)
    if b.out.shape[1:] != (hidden,):
        raise ValueError(f"buffers.out: shape {tuple(b.out.shape)}, expected [T, {hidden}]")
    _workspace(b.workspace, x.device, stream)
    rc = load().moe_layer_forward_fp4(
        _ptr(x), _ptr(topk_ids), _ptr(topk_w), T, k, E, hidden, inter, fmt, _ptr(c13), _ptr(s13),
        _tensor_scale("w13 weight_scale_2", g13, E, fmt), _ptr(c2), _ptr(s2),
        _tensor_scale("w2 weight_scale_2", g2, E, fmt), _tensor_scale("x_scale_2", x_scale_2, 1, fmt),
        _tensor_scale("h_scale_2", h_scale_2, 1, fmt), _ptr(b.out), _ptr(b.group_sizes),
        _ptr(b.group_offsets), _ptr(b.sorted_slot), _ptr(b.slot_to_row), _ptr(b.x_codes),
        _ptr(b.x_scales), _ptr(b.h_codes), _ptr(b.h_scales), _ptr(b.y2), _ptr(b.workspace),
        b.workspace.numel(), _stream(stream))
    _check(rc, "moe_layer_forward_fp4")
    return b.out if b.out.shape[0] == T else b.out[:T]


def debug_bounded_wait(limit_ns: int, workspace: torch.Tensor, stream=None):
    rc = load().moe_debug_bounded_wait(int(limit_ns), _ptr(workspace), workspace.numel(),
                                       _stream(stream))
    _check(rc, "moe_debug_bounded_wait")


# ---------------------------------------------------------------- marshalling

def bf16_from_bits(bits, device="cuda") -> torch.Tensor:
    """numpy uint16 bf16 patterns -> device bf16 tensor (bit-exact)."""
    import numpy as np
    a = np.ascontiguousarray(bits, dtype=np.uint16).view(np.int16)
    return torch.from_numpy(a).to(device).view(torch.bfloat16)


def bits_from_bf16(t: torch.Tensor):
    """device bf16 tensor -> numpy uint16 bit patterns."""
    import numpy as np
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def to_device(a, device="cuda") -> torch.Tensor:
    import numpy as np
    return torch.from_numpy(np.ascontiguousarray(a)).to(device)
