"""Switch Transformer sparse FFN layer forward pass on NVIDIA B200 (sm_100a).

Python binding of the C ABI in ``include/switch_moe.h``.  It only marshals
arguments: every step of the layer runs in the CUDA kernels of
``libswitchmoe.so``, which this module loads from the package directory.
There is no other implementation behind these functions; if the library is
missing or cannot be loaded, every call raises.

PyTorch supplies device memory and the CUDA stream (the current stream of the
tensors' device unless one is given).

Low level (same names and argument order as the C functions, tensors in
place of pointers):
    switch_capacity, switch_workspace_size, switch_route, switch_dispatch,
    switch_expert_ffn, switch_combine, switch_layer_fwd, switch_check
High level (allocate outputs and workspace with torch):
    capacity, layer_fwd, layer_bwd, layer_fwd_top2, route, route_top2, router_stats
    norm_fwd, norm_bwd      the residual's addition with its root-mean-square norm, and its gradient
    quantize_rows           rows in 8 bits with scales
    FewLayer, layer_fwd_few the whole layer for a few tokens (float32, bfloat16 or 8-bit experts)
    block_fwd, block_bwd    residual and norm, then the layer
"""
from __future__ import annotations

import ctypes
import functools
import operator
from pathlib import Path

_PKG = Path(__file__).resolve().parent
LIB_PATH = _PKG / "libswitchmoe.so"

SWITCH_F32 = 0
SWITCH_BF16 = 1
SWITCH_E4M3 = 2
SWITCH_FEW_MAX_TOKENS = 64
SWITCH_FLAG_SIMT_FFN = 1
SWITCH_FLAG_SIMT_ROUTER = 2
SWITCH_FLAG_GEMM_1CTA = 4
SWITCH_FLAG_FFN_TWO_LAUNCHES = 8
SWITCH_FLAG_SEPARATE_SCAN = 16
SWITCH_FLAG_TRAINING = 32
SWITCH_FLAG_ROUTER_STATS = 64
SWITCH_FLAG_MULTI_KERNEL = 128
SWITCH_FLAG_STAGED_MOVES = 256

STATUS = {
    0: "SWITCH_OK", 1: "SWITCH_ERR_NULL", 2: "SWITCH_ERR_SHAPE", 3: "SWITCH_ERR_DTYPE", 4: "SWITCH_ERR_ALIGN",
    5: "SWITCH_ERR_WORKSPACE", 6: "SWITCH_ERR_UNSUPPORTED", 7: "SWITCH_ERR_CUDA", 8: "SWITCH_ERR_DEVICE_TIMEOUT",
    9: "SWITCH_ERR_TOO_LARGE",
}

EXPORTED = ("switch_capacity", "switch_workspace_size", "switch_route", "switch_route_noalloc", "switch_dispatch",
            "switch_expert_ffn",
            "switch_combine", "switch_layer_fwd", "switch_route_top2", "switch_combine_top2", "switch_layer_fwd_top2",
            "switch_layer_bwd", "switch_router_stats",
            "switch_few_workspace_size", "switch_layer_fwd_few", "switch_norm_fwd", "switch_norm_workspace_size",
            "switch_norm_bwd", "switch_quantize_rows",
            "switch_check", "switch_selftest_wait_timeout", "switch_check_noalloc",
            "switch_selftest_wait_timeout_noalloc", "switch_status_string",
            "switch_launch_count",
            "switch_trace_start", "switch_trace_read", "switch_trace_stop", "switch_kernel_name")


class SwitchError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} ({_status_text(status)})")


class SwitchDims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("d_model", ctypes.c_int32), ("d_ff", ctypes.c_int32),
                ("num_experts", ctypes.c_int32), ("capacity", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("flags", ctypes.c_int32)]

    def __repr__(self):
        return (f"SwitchDims(T={self.T}, d_model={self.d_model}, d_ff={self.d_ff}, num_experts={self.num_experts}, "
                f"capacity={self.capacity}, dtype={self.dtype}, flags={self.flags})")


class SwitchNormDims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("d_model", ctypes.c_int32), ("residual_dtype", ctypes.c_int32),
                ("delta_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("eps", ctypes.c_float)]

    def __repr__(self):
        return (f"SwitchNormDims(T={self.T}, d_model={self.d_model}, residual_dtype={self.residual_dtype}, "
                f"delta_dtype={self.delta_dtype}, out_dtype={self.out_dtype}, eps={self.eps})")


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded CUDA library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not LIB_PATH.exists():
        raise RuntimeError(f"{LIB_PATH.name} is not built; run `python -m sparse_mixture_experts_fp32_b200.build`")
    L = ctypes.CDLL(str(LIB_PATH))
    P, S = ctypes.c_void_p, ctypes.c_size_t
    D = ctypes.POINTER(SwitchDims)
    ND = ctypes.POINTER(SwitchNormDims)
    I = ctypes.c_int
    sig = {
        "switch_capacity": (ctypes.c_int64, [ctypes.c_int64, ctypes.c_int32, ctypes.c_double]),
        "switch_workspace_size": (I, [D, ctypes.POINTER(ctypes.c_size_t)]),
        "switch_route": (I, [D, P, P, P, P, P, P, P, P, P, P, S, P]),
        "switch_route_noalloc": (I, [D, P, P, P, P, P, P, P, P, P, P]),
        "switch_dispatch": (I, [D, P, P, P, P, P]),
        "switch_expert_ffn": (I, [D, P, P, P, P, P, P, S, P]),
        "switch_combine": (I, [D, P, P, P, P, P, P]),
        "switch_layer_fwd": (I, [D, P, P, P, P, P, P, P, P, P, P, P, P, S, P]),
        "switch_route_top2": (I, [D, P, P, P, P, P, P, P, P, P, P, S, P]),
        "switch_combine_top2": (I, [D, P, P, P, P, P, P]),
        "switch_layer_fwd_top2": (I, [D, P, P, P, P, P, P, P, P, P, P, P, P, S, P]),
        "switch_layer_bwd": (I, [D, P, P, P, P, P, P, P, P, P, ctypes.c_float, P, P, P, P, P, P, S, P]),
        "switch_router_stats": (I, [D, P, P, S, P, P]),
        "switch_few_workspace_size": (I, [D, ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)]),
        "switch_layer_fwd_few": (I, [D, ctypes.c_int32] + [P] * 15 + [S, P]),
        "switch_norm_fwd": (I, [ND, P, P, P, P, P, P, P, P]),
        "switch_norm_workspace_size": (I, [ND, ctypes.POINTER(ctypes.c_size_t)]),
        "switch_norm_bwd": (I, [ND, P, P, P, P, P, P, P, P, S, P]),
        "switch_quantize_rows": (I, [ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, P, P, P, P]),
        "switch_check": (I, [P, S, P]),
        "switch_selftest_wait_timeout": (I, [P, S, P]),
        "switch_check_noalloc": (I, [P]),
        "switch_selftest_wait_timeout_noalloc": (I, [P]),
        "switch_status_string": (ctypes.c_char_p, [I]),
        "switch_launch_count": (ctypes.c_int64, []),
        "switch_trace_start": (I, [ctypes.c_int32]),
        "switch_trace_read": (ctypes.c_int32, [P, P, ctypes.c_int32]),
        "switch_trace_stop": (None, []),
        "switch_kernel_name": (ctypes.c_char_p, [ctypes.c_int32]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _lib = L
    return L


def _status_text(status: int) -> str:
    try:
        return lib().switch_status_string(status).decode()
    except Exception:
        return "?"


def _ok(status: int, where: str) -> None:
    if status != 0:
        raise SwitchError(status, where)


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------
def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise TypeError("switch_moe tensors must be CUDA tensors")
    if not t.is_contiguous():
        raise TypeError("switch_moe tensors must be contiguous")
    return t.data_ptr()


def _stream(stream, like=None):
    import torch
    if stream is None:
        dev = like.device if like is not None and hasattr(like, "device") else None
        return torch.cuda.current_stream(dev).cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def dtype_code(dtype) -> int:
    import torch
    if dtype == torch.float32:
        return SWITCH_F32
    if dtype == torch.bfloat16:
        return SWITCH_BF16
    raise TypeError(f"activations and expert weights must be float32 or bfloat16, got {dtype}")


def dims(T: int, d_model: int, d_ff: int, num_experts: int, capacity: int, dtype, flags: int = 0) -> SwitchDims:
    code = dtype if isinstance(dtype, int) else dtype_code(dtype)
    return SwitchDims(int(T), int(d_model), int(d_ff), int(num_experts), int(capacity), code, int(flags))


# ---------------------------------------------------------------------------
# low level: the C functions
# ---------------------------------------------------------------------------
def switch_capacity(T: int, num_experts: int, capacity_factor: float) -> int:
    return int(lib().switch_capacity(int(T), int(num_experts), float(capacity_factor)))


def switch_workspace_size(d: SwitchDims) -> int:
    out = ctypes.c_size_t(0)
    _ok(lib().switch_workspace_size(ctypes.byref(d), ctypes.byref(out)), "switch_workspace_size")
    return int(out.value)


def switch_route(d, x, w_r, logit_bias, expert, gate, slot, counts, slot_token, aux, workspace, stream=None):
    _ok(lib().switch_route(ctypes.byref(d), _ptr(x), _ptr(w_r), _ptr(logit_bias), _ptr(expert), _ptr(gate),
                           _ptr(slot), _ptr(counts), _ptr(slot_token), _ptr(aux), _ptr(workspace),
                           workspace.numel() * workspace.element_size(), _stream(stream, workspace)),
        "switch_route")


def switch_route_noalloc(d, x, w_r, logit_bias, expert, gate, slot, counts, slot_token, aux, stream=None):
    """switch_route without a workspace: for callers that cannot allocate
    device memory where they route (the scratch is a static array inside the
    library; calls that overlap on the GPU race)."""
    _ok(lib().switch_route_noalloc(ctypes.byref(d), _ptr(x), _ptr(w_r), _ptr(logit_bias), _ptr(expert), _ptr(gate),
                                   _ptr(slot), _ptr(counts), _ptr(slot_token), _ptr(aux), _stream(stream, counts)),
        "switch_route_noalloc")


def switch_dispatch(d, x, slot_token, counts, xbuf, stream=None):
    _ok(lib().switch_dispatch(ctypes.byref(d), _ptr(x), _ptr(slot_token), _ptr(counts), _ptr(xbuf),
                              _stream(stream, xbuf)), "switch_dispatch")


def switch_expert_ffn(d, xbuf, w_in, w_out, counts, ybuf, workspace, stream=None):
    _ok(lib().switch_expert_ffn(ctypes.byref(d), _ptr(xbuf), _ptr(w_in), _ptr(w_out), _ptr(counts), _ptr(ybuf),
                                _ptr(workspace), workspace.numel() * workspace.element_size(),
                                _stream(stream, workspace)), "switch_expert_ffn")


def switch_combine(d, ybuf, expert, slot, gate, y, stream=None):
    _ok(lib().switch_combine(ctypes.byref(d), _ptr(ybuf), _ptr(expert), _ptr(slot), _ptr(gate), _ptr(y),
                             _stream(stream, ybuf)), "switch_combine")


def switch_layer_fwd(d, x, w_r, logit_bias, w_in, w_out, y, expert, gate, slot, counts, aux, workspace, stream=None):
    _ok(lib().switch_layer_fwd(ctypes.byref(d), _ptr(x), _ptr(w_r), _ptr(logit_bias), _ptr(w_in), _ptr(w_out),
                               _ptr(y), _ptr(expert), _ptr(gate), _ptr(slot), _ptr(counts), _ptr(aux),
                               _ptr(workspace), workspace.numel() * workspace.element_size(),
                               _stream(stream, workspace)), "switch_layer_fwd")


def switch_route_top2(d, x, w_r, logit_bias, expert, gate, slot, counts, slot_token, aux, workspace, stream=None):
    _ok(lib().switch_route_top2(ctypes.byref(d), _ptr(x), _ptr(w_r), _ptr(logit_bias), _ptr(expert), _ptr(gate),
                                _ptr(slot), _ptr(counts), _ptr(slot_token), _ptr(aux), _ptr(workspace),
                                workspace.numel() * workspace.element_size(), _stream(stream, workspace)),
        "switch_route_top2")


def switch_combine_top2(d, ybuf, expert, slot, gate, y, stream=None):
    _ok(lib().switch_combine_top2(ctypes.byref(d), _ptr(ybuf), _ptr(expert), _ptr(slot), _ptr(gate), _ptr(y),
                                  _stream(stream, ybuf)), "switch_combine_top2")


def switch_layer_fwd_top2(d, x, w_r, logit_bias, w_in, w_out, y, expert, gate, slot, counts, aux, workspace,
                          stream=None):
    _ok(lib().switch_layer_fwd_top2(ctypes.byref(d), _ptr(x), _ptr(w_r), _ptr(logit_bias), _ptr(w_in), _ptr(w_out),
                                    _ptr(y), _ptr(expert), _ptr(gate), _ptr(slot), _ptr(counts), _ptr(aux),
                                    _ptr(workspace), workspace.numel() * workspace.element_size(),
                                    _stream(stream, workspace)), "switch_layer_fwd_top2")


def switch_layer_bwd(d, x, w_r, w_in, w_out, expert, gate, slot, counts, dy, g_aux, dx, dw_r, dbias, dw_in, dw_out,
                     workspace, stream=None):
    _ok(lib().switch_layer_bwd(ctypes.byref(d), _ptr(x), _ptr(w_r), _ptr(w_in), _ptr(w_out), _ptr(expert),
                               _ptr(gate), _ptr(slot), _ptr(counts), _ptr(dy), float(g_aux), _ptr(dx), _ptr(dw_r),
                               _ptr(dbias), _ptr(dw_in), _ptr(dw_out), _ptr(workspace),
                               workspace.numel() * workspace.element_size(), _stream(stream, workspace)),
        "switch_layer_bwd")


def switch_router_stats(d, counts, workspace, stats, stream=None):
    _ok(lib().switch_router_stats(ctypes.byref(d), _ptr(counts), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), _ptr(stats),
                                  _stream(stream, workspace)), "switch_router_stats")


def switch_few_workspace_size(d: SwitchDims, top_k: int) -> int:
    out = ctypes.c_size_t(0)
    _ok(lib().switch_few_workspace_size(ctypes.byref(d), int(top_k), ctypes.byref(out)), "switch_few_workspace_size")
    return int(out.value)


def switch_layer_fwd_few(d, top_k, x, x_scale, w_r, logit_bias, w_in, w_in_scale, w_out, w_out_scale, y, expert, gate,
                         slot, counts, aux, workspace, stream=None):
    _ok(lib().switch_layer_fwd_few(ctypes.byref(d), int(top_k), _ptr(x), _ptr(x_scale), _ptr(w_r), _ptr(logit_bias),
                                   _ptr(w_in), _ptr(w_in_scale), _ptr(w_out), _ptr(w_out_scale), _ptr(y),
                                   _ptr(expert), _ptr(gate), _ptr(slot), _ptr(counts), _ptr(aux), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), _stream(stream, workspace)),
        "switch_layer_fwd_few")


def switch_norm_fwd(d, residual, delta, weight, sum, out, scale, rstd, stream=None):
    _ok(lib().switch_norm_fwd(ctypes.byref(d), _ptr(residual), _ptr(delta), _ptr(weight), _ptr(sum), _ptr(out),
                              _ptr(scale), _ptr(rstd), _stream(stream, out)), "switch_norm_fwd")


def switch_norm_workspace_size(d: SwitchNormDims) -> int:
    out = ctypes.c_size_t(0)
    _ok(lib().switch_norm_workspace_size(ctypes.byref(d), ctypes.byref(out)), "switch_norm_workspace_size")
    return int(out.value)


def switch_norm_bwd(d, sum, weight, rstd, dout, dsum, dresidual, dweight, workspace, stream=None):
    _ok(lib().switch_norm_bwd(ctypes.byref(d), _ptr(sum), _ptr(weight), _ptr(rstd), _ptr(dout), _ptr(dsum),
                              _ptr(dresidual), _ptr(dweight), _ptr(workspace),
                              workspace.numel() * workspace.element_size(), _stream(stream, workspace)),
        "switch_norm_bwd")


def switch_quantize_rows(rows, cols, dtype, x, q, scale, stream=None):
    code = dtype if isinstance(dtype, int) else dtype_code(dtype)
    _ok(lib().switch_quantize_rows(int(rows), int(cols), code, _ptr(x), _ptr(q), _ptr(scale), _stream(stream, q)),
        "switch_quantize_rows")


def switch_check(workspace, stream=None) -> int:
    """Synchronise and return the device status code (0 = ok); does not raise."""
    return int(lib().switch_check(_ptr(workspace), workspace.numel() * workspace.element_size(),
                                  _stream(stream, workspace)))


def selftest_wait_timeout(workspace, stream=None) -> None:
    """Launch the bounded-wait self-test; switch_check(workspace) afterwards
    reports SWITCH_ERR_DEVICE_TIMEOUT (8)."""
    _ok(lib().switch_selftest_wait_timeout(_ptr(workspace), workspace.numel() * workspace.element_size(),
                                           _stream(stream, workspace)), "switch_selftest_wait_timeout")


def switch_check_noalloc(stream=None) -> int:
    """switch_check for the static array switch_route_noalloc uses (0 = ok); does not raise."""
    return int(lib().switch_check_noalloc(_stream(stream)))


def selftest_wait_timeout_noalloc(stream=None) -> None:
    """The bounded-wait self-test on the static routing array's status word."""
    _ok(lib().switch_selftest_wait_timeout_noalloc(_stream(stream)), "switch_selftest_wait_timeout_noalloc")


def launch_count() -> int:
    return int(lib().switch_launch_count())


def trace_start(max_launches: int) -> None:
    _ok(lib().switch_trace_start(int(max_launches)), "switch_trace_start")


def trace_read(capacity: int = 4096) -> list[tuple[str, float]]:
    ids = (ctypes.c_int32 * capacity)()
    ms = (ctypes.c_float * capacity)()
    n = lib().switch_trace_read(ids, ms, capacity)
    return [(lib().switch_kernel_name(ids[k]).decode(), float(ms[k])) for k in range(n)]


def trace_stop() -> None:
    lib().switch_trace_stop()


# ---------------------------------------------------------------------------
# high level: torch-allocating wrappers
# ---------------------------------------------------------------------------
def capacity(T: int, num_experts: int, capacity_factor: float) -> int:
    c = switch_capacity(T, num_experts, capacity_factor)
    if c < 1:
        raise ValueError("capacity needs T >= 0, num_experts >= 1 and a positive capacity factor")
    return c


def _resolve_capacity(T, N, cap, capacity_factor):
    if cap is not None:
        return int(cap)
    if capacity_factor is None:
        raise ValueError("give capacity or capacity_factor")
    c = switch_capacity(T, N, capacity_factor)
    if c < 1:
        raise ValueError("capacity needs T >= 0, num_experts >= 1 and a positive capacity factor")
    return c


def workspace(d: SwitchDims, device):
    import torch
    return torch.empty(switch_workspace_size(d), dtype=torch.uint8, device=device)


def layer_dims(x, w_in, capacity=None, capacity_factor=None, flags: int = 0) -> SwitchDims:
    T, dm = x.shape
    N, F, dm2 = w_in.shape
    if dm2 != dm:
        raise ValueError("w_in must be [N, d_ff, d_model]")
    if w_in.dtype != x.dtype:
        raise TypeError("x and the expert weights must share a dtype")
    C = _resolve_capacity(T, N, capacity, capacity_factor)
    return dims(T, dm, F, N, C, x.dtype, flags)


def layer_fwd(x, w_r, w_in, w_out, capacity=None, capacity_factor=None, logit_bias=None, flags: int = 0,
              ws=None, out=None, stream=None):
    """The Switch layer forward pass.  Returns a dict with y [T, d] float32
    (no residual), aux (1-element float32), expert, gate, slot, counts."""
    import torch
    d = layer_dims(x, w_in, capacity, capacity_factor, flags)
    T, dev = x.shape[0], x.device
    if out is None:
        out = dict(y=torch.empty(x.shape, dtype=torch.float32, device=dev), expert=torch.empty(T, dtype=torch.int32, device=dev),
                   gate=torch.empty(T, dtype=torch.float32, device=dev),
                   slot=torch.empty(T, dtype=torch.int32, device=dev),
                   counts=torch.empty(d.num_experts, dtype=torch.int32, device=dev),
                   aux=torch.empty(1, dtype=torch.float32, device=dev))
    if ws is None:
        ws = workspace(d, dev)
    switch_layer_fwd(d, x, w_r, logit_bias, w_in, w_out, out["y"], out["expert"], out["gate"], out["slot"],
                     out["counts"], out["aux"], ws, stream)
    out["capacity"] = d.capacity
    out["flags"] = d.flags
    out["workspace"] = ws
    return out


def route(x, w_r, num_experts=None, capacity=None, capacity_factor=None, logit_bias=None, d_ff: int = 64,
          ws=None, stream=None, flags: int = 0):
    """Router, top-1, capacity assignment, counts and aux (switch_route)."""
    import torch
    T, dm = x.shape
    N = w_r.shape[0] if num_experts is None else num_experts
    C = _resolve_capacity(T, N, capacity, capacity_factor)
    d = dims(T, dm, d_ff, N, C, x.dtype, flags)
    dev = x.device
    out = dict(expert=torch.empty(T, dtype=torch.int32, device=dev),
               gate=torch.empty(T, dtype=torch.float32, device=dev),
               slot=torch.empty(T, dtype=torch.int32, device=dev),
               counts=torch.empty(N, dtype=torch.int32, device=dev),
               slot_token=torch.empty(N * C, dtype=torch.int32, device=dev),
               aux=torch.empty(1, dtype=torch.float32, device=dev))
    if ws is None:
        ws = workspace(d, dev)
    switch_route(d, x, w_r, logit_bias, out["expert"], out["gate"], out["slot"], out["counts"], out["slot_token"],
                 out["aux"], ws, stream)
    out["capacity"] = C
    out["flags"] = d.flags
    out["workspace"] = ws
    return out


def layer_fwd_top2(x, w_r, w_in, w_out, capacity=None, capacity_factor=None, logit_bias=None, flags: int = 0,
                   ws=None, out=None, stream=None):
    """The top-2 mixture-of-experts layer forward pass.  Returns a dict with
    y [T, d] float32, aux, expert / gate / slot [T, 2], counts [N]."""
    import torch
    d = layer_dims(x, w_in, capacity, capacity_factor, flags)
    T, dev = x.shape[0], x.device
    if out is None:
        out = dict(y=torch.empty(x.shape, dtype=torch.float32, device=dev),
                   expert=torch.empty(T, 2, dtype=torch.int32, device=dev),
                   gate=torch.empty(T, 2, dtype=torch.float32, device=dev),
                   slot=torch.empty(T, 2, dtype=torch.int32, device=dev),
                   counts=torch.empty(d.num_experts, dtype=torch.int32, device=dev),
                   aux=torch.empty(1, dtype=torch.float32, device=dev))
    if ws is None:
        ws = workspace(d, dev)
    switch_layer_fwd_top2(d, x, w_r, logit_bias, w_in, w_out, out["y"], out["expert"], out["gate"], out["slot"],
                          out["counts"], out["aux"], ws, stream)
    out["capacity"] = d.capacity
    out["workspace"] = ws
    return out


def route_top2(x, w_r, capacity=None, capacity_factor=None, logit_bias=None, d_ff: int = 64, ws=None, stream=None,
               flags: int = 0):
    """Router, top-2, capacity assignment, counts and aux (switch_route_top2)."""
    import torch
    T, dm = x.shape
    N = w_r.shape[0]
    C = _resolve_capacity(T, N, capacity, capacity_factor)
    d = dims(T, dm, d_ff, N, C, x.dtype, flags)
    dev = x.device
    out = dict(expert=torch.empty(T, 2, dtype=torch.int32, device=dev),
               gate=torch.empty(T, 2, dtype=torch.float32, device=dev),
               slot=torch.empty(T, 2, dtype=torch.int32, device=dev),
               counts=torch.empty(N, dtype=torch.int32, device=dev),
               slot_token=torch.empty(N * C, dtype=torch.int32, device=dev),
               aux=torch.empty(1, dtype=torch.float32, device=dev))
    if ws is None:
        ws = workspace(d, dev)
    switch_route_top2(d, x, w_r, logit_bias, out["expert"], out["gate"], out["slot"], out["counts"],
                      out["slot_token"], out["aux"], ws, stream)
    out["capacity"] = C
    out["flags"] = d.flags
    out["workspace"] = ws
    return out


def layer_bwd(fwd: dict, x, w_r, w_in, w_out, dy, g_aux: float = 0.0, logit_bias=None, stream=None):
    """Gradients of sum(y * dy) + g_aux * aux after ``layer_fwd(..., flags=SWITCH_FLAG_TRAINING)``
    (whose result dict, with its workspace, is ``fwd``; a top-2 forward has no backward pass).
    Returns dx, dw_r, dbias (None without a logit bias), dw_in, dw_out, all float32."""
    import torch
    T, dm = x.shape
    if tuple(fwd["expert"].shape) != (T,):
        raise ValueError(f"fwd must be layer_fwd's result for x, one expert per token: expert is "
                         f"{list(fwd['expert'].shape)} for {T} tokens")
    N, F, _ = w_in.shape
    dev = x.device
    d = layer_dims(x, w_in, capacity=fwd["capacity"], flags=fwd.get("flags", SWITCH_FLAG_TRAINING))
    out = dict(dx=torch.empty(T, dm, dtype=torch.float32, device=dev),
               dw_r=torch.empty(N, dm, dtype=torch.float32, device=dev),
               dbias=torch.empty(N, dtype=torch.float32, device=dev) if logit_bias is not None else None,
               dw_in=torch.empty(N, F, dm, dtype=torch.float32, device=dev),
               dw_out=torch.empty(N, dm, F, dtype=torch.float32, device=dev))
    switch_layer_bwd(d, x, w_r, w_in, w_out, fwd["expert"], fwd["gate"], fwd["slot"], fwd["counts"], dy, g_aux,
                     out["dx"], out["dw_r"], out["dbias"], out["dw_in"], out["dw_out"], fwd["workspace"], stream)
    return out


def router_stats(result: dict, T: int, d_model: int, d_ff: int, dtype, stream=None):
    """Router statistics of a route / layer_fwd result made with SWITCH_FLAG_ROUTER_STATS:
    a 4-element float32 tensor (mean entropy, dropped fraction, capacity utilisation, busiest load)."""
    import torch
    counts = result["counts"]
    d = dims(T, d_model, d_ff, counts.numel(), result["capacity"], dtype, result.get("flags", SWITCH_FLAG_ROUTER_STATS))
    stats = torch.empty(4, dtype=torch.float32, device=counts.device)
    switch_router_stats(d, counts, result["workspace"], stats, stream)
    return stats


# ---------------------------------------------------------------------------
# residual + norm, 8-bit rows, the layer for a few tokens
# ---------------------------------------------------------------------------
class _Names:
    """What the calls below need of torch, looked up once: a call of theirs is about as long as its Python."""

    def __init__(self):
        import torch
        self.torch = torch
        self.codes = {torch.float32: SWITCH_F32, torch.bfloat16: SWITCH_BF16, torch.float8_e4m3fn: SWITCH_E4M3}
        self.f32, self.e4m3 = (torch.float32,), torch.float8_e4m3fn
        self.floats = (torch.float32, torch.bfloat16)
        self.current_device = torch.cuda.current_device
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # without a torch.cuda.Stream around it (2 us)
        self.current_stream = raw if raw is not None else lambda i: torch.cuda.current_stream(i).cuda_stream


_names = None


def _torch_names() -> _Names:
    global _names
    if _names is None:
        _names = _Names()
    return _names


def _code(dtype) -> int:
    """dtype_code with the 8-bit type (which only the calls below take)."""
    code = (_names or _torch_names()).codes.get(dtype)
    return dtype_code(dtype) if code is None else code


def _want(name, t, shape, dtypes, device):
    """Checks an argument and returns its pointer (None for None)."""
    if t is None:
        return None
    if t.shape == shape and t.dtype in dtypes and t.device == device and t.is_contiguous() and t.is_cuda:
        return t.data_ptr()
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    return _ptr(t)


class _Result(dict):
    """A result that a later call of the same sizes may write into again (out=): the tensors of its first call,
    whatever the dict holds by then.  They may not be inputs of that call, other than where it says so."""
    __slots__ = ("key", "own", "addresses")

    def holds(self, *inputs):
        """Whether one of the inputs' addresses is one of the tensors'."""
        if self.addresses is None:
            self.addresses = frozenset(t.data_ptr() for t in self.own.values() if t is not None)
        return not self.addresses.isdisjoint(inputs)

    def refuse(self, **inputs):
        """Raises where an input is one of the tensors."""
        for name, address in inputs.items():
            if address and address in self.addresses:
                raise ValueError(f"{name} is a tensor of the result given as out, which the call overwrites")


def _result(out, key, make):
    """`out` when it came from a call with the same `key`, else new outputs (out=None) or an error."""
    if out is None:
        own = make()
        out = _Result(own)
        out.key, out.own, out.addresses = key, own, None
    elif type(out) is not _Result or out.key != key:
        raise ValueError("out must be the result of an earlier call of the same function, sizes, types and device")
    else:
        out.update(out.own)
    return out


def _launch(fn, where, device, *args):
    """Calls the C function on the current stream of `device`, which is made current meanwhile."""
    z, index = _names, device.index
    if z.current_device() == index:
        status = fn(*args, z.current_stream(index))
    else:
        with z.torch.cuda.device(device):
            status = fn(*args, z.current_stream(index))
    if status != 0:
        raise SwitchError(status, where)


def _under(stream, device):
    """Makes `stream` (a torch stream or a cudaStream_t) the current one, so that what is allocated meanwhile is
    ordered on the stream that it is used on."""
    import torch
    if not isinstance(stream, int) and stream.device != device:
        raise ValueError(f"stream must be on {device}, got {stream.device}")
    return torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device) if isinstance(stream, int) else stream)


def _current(device):
    """Makes `device` the current one, for the calls that go by it (those above do so themselves)."""
    import torch
    return torch.cuda.device(device)


def _rows(name, t):
    """Shape and device of a [rows, columns] CUDA tensor."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be [rows, columns], got {list(shape)}")
    if not t.is_cuda:
        raise TypeError("switch_moe tensors must be CUDA tensors")
    return shape, t.device


def norm_fwd(residual, weight, delta=None, eps: float = 1e-6, out_dtype=None, inplace: bool = False, out=None,
             stream=None):
    """s = residual + delta, rounded to residual's type, and out = s / rms(s) * weight (switch_norm_fwd).

    residual [T, d] float32 or bfloat16; delta [T, d] float32 or bfloat16 (a layer's y), or None for s = residual;
    weight [d] float32; out_dtype float32, bfloat16 or float8_e4m3fn (default: residual's).  Returns a dict with
    sum (None without a delta; residual itself with ``inplace``, which delta may then not overlap), out, scale ([T],
    8-bit outputs only) and rstd [T].
    ``out`` takes the result of an earlier call of the same sizes, which is overwritten: no input may be a part of
    it, but its sum may be residual."""
    shape, dev = _rows("residual", residual)
    if stream is not None:
        with _under(stream, dev):
            return norm_fwd(residual, weight, delta, eps, out_dtype, inplace, out)
    z = _names or _torch_names()
    T, dm = shape
    dtype = residual.dtype
    if out_dtype is None:
        out_dtype = dtype
    out_code = _code(out_dtype)
    pr, pd = _want("residual", residual, shape, z.floats, dev), _want("delta", delta, shape, z.floats, dev)
    pw = _want("weight", weight, (dm,), z.f32, dev)
    stored = delta is not None and not inplace
    key = ("norm_fwd", shape, dtype, out_dtype, stored, dev)
    reuse = out is not None
    if not reuse or type(out) is not _Result or out.key != key:
        empty, f32 = z.torch.empty, z.torch.float32
        out = _result(out, key, lambda: dict(
            sum=z.torch.empty_like(residual) if stored else None, out=empty(shape, dtype=out_dtype, device=dev),
            scale=empty(T, dtype=f32, device=dev) if out_dtype == z.e4m3 else None,
            rstd=empty(T, dtype=f32, device=dev)))
    own = out.own
    total, scale, codes = own["sum"], own["scale"], z.codes
    if reuse and out.holds(pr, pd, pw):  # sum may be residual itself
        out.refuse(residual=None if total is not None and pr == total.data_ptr() else pr, delta=pd, weight=pw)
    out.update(own)
    if total is not None:
        ps = total.data_ptr()
    elif delta is not None:
        out["sum"], ps = residual, pr
    else:
        ps = None
    d = SwitchNormDims(T, dm, codes[dtype], SWITCH_F32 if delta is None else codes[delta.dtype],
                       out_code, eps)
    _launch(lib().switch_norm_fwd, "switch_norm_fwd", dev, ctypes.byref(d), pr, pd, pw, ps, own["out"].data_ptr(),
            None if scale is None else scale.data_ptr(), own["rstd"].data_ptr())
    return out


@functools.lru_cache(maxsize=64)
def _norm_bwd_dims(T, d_model, code):
    d = SwitchNormDims(T, d_model, code, SWITCH_F32, SWITCH_F32, 0.0)
    return d, ctypes.byref(d), switch_norm_workspace_size(d)


def norm_bwd(sum, weight, rstd, dout, dsum=None, out=None, stream=None):
    """Gradient of norm_fwd (switch_norm_bwd): from dout [T, d] float32 (the gradient of its out) and dsum [T, d]
    float32 (the gradient of its sum from elsewhere, or None), dresidual [T, d] (of residual and of delta alike) and
    dweight [d], float32.  sum is norm_fwd's sum, or residual where there was no delta.  ``out`` takes the result of
    an earlier call of the same sizes, which is overwritten: its dresidual may be dout or dsum, no other input a part
    of it."""
    shape, dev = _rows("sum", sum)
    if stream is not None:
        with _under(stream, dev):
            return norm_bwd(sum, weight, rstd, dout, dsum, out)
    z = _names or _torch_names()
    T, dm = shape
    f32 = z.f32
    ps, pw = _want("sum", sum, shape, z.floats, dev), _want("weight", weight, (dm,), f32, dev)
    pr, pg, pu = (_want("rstd", rstd, (T,), f32, dev), _want("dout", dout, shape, f32, dev),
                  _want("dsum", dsum, shape, f32, dev))
    empty, reuse = z.torch.empty, out is not None
    out = _result(out, ("norm_bwd", shape, dev), lambda: dict(
        dresidual=empty(shape, dtype=f32[0], device=dev), dweight=empty(dm, dtype=f32[0], device=dev)))
    own = out.own
    if reuse and out.holds(ps, pw, pr, pg, pu):
        at = own["dresidual"].data_ptr()
        out.refuse(sum=ps, weight=pw, rstd=pr, dout=None if pg == at else pg, dsum=None if pu == at else pu)
    _, ref, size = _norm_bwd_dims(T, dm, z.codes[sum.dtype])
    ws = empty(size, dtype=z.torch.uint8, device=dev)
    _launch(lib().switch_norm_bwd, "switch_norm_bwd", dev, ref, ps, pw, pr, pg, pu,
            own["dresidual"].data_ptr(), own["dweight"].data_ptr(), ws.data_ptr(), size)
    return out


def quantize_rows(x, out=None, stream=None):
    """x [..., cols] float32 or bfloat16 in 8 bits (switch_quantize_rows): a dict with q (float8_e4m3fn, x's shape)
    and scale (float32, x's shape without the last dimension); x is about q * scale.  ``out`` takes the result of an
    earlier call of the same sizes, which is overwritten: x may not be a part of it."""
    if not x.is_cuda:
        raise TypeError("switch_moe tensors must be CUDA tensors")
    shape, dev = x.shape, x.device
    if len(shape) < 1:
        raise ValueError("x must have rows")
    if stream is not None:
        with _under(stream, dev):
            return quantize_rows(x, out)
    z = _names or _torch_names()
    rows = 1
    for n in shape[:-1]:
        rows *= n
    px = _want("x", x, shape, z.floats, dev)
    empty, reuse = z.torch.empty, out is not None
    out = _result(out, ("quantize_rows", shape, dev), lambda: dict(
        q=empty(shape, dtype=z.e4m3, device=dev), scale=empty(shape[:-1], dtype=z.torch.float32, device=dev)))
    own = out.own
    if reuse and out.holds(px):
        out.refuse(x=px)
    _launch(lib().switch_quantize_rows, "switch_quantize_rows", dev, rows, shape[-1], z.codes[x.dtype], px,
            own["q"].data_ptr(), own["scale"].data_ptr())
    return out


class FewLayer:
    """The layer for up to 64 tokens over one set of weights (switch_layer_fwd_few): the handle that a serving
    program keeps.  w_r [N, d] float32; w_in [N, F, d] and w_out [N, d, F] float32, bfloat16 or float8_e4m3fn, the
    last with w_in_scale [N, F] and w_out_scale [N, d] (quantize_rows makes both).  ``capacity`` None keeps every
    token.  The tensors are held and read at each call, so they may be updated in place; the handle's attributes
    cannot be set (other sizes, weights or a capacity are another handle).  Calls may run on several streams at once
    (each has a workspace of its own unless it is given one)."""

    def __init__(self, w_r, w_in, w_out, top_k: int = 1, capacity=None, capacity_factor=None, logit_bias=None,
                 w_in_scale=None, w_out_scale=None, flags: int = 0):
        import torch
        if w_in.dim() != 3:
            raise ValueError("w_in must be [N, d_ff, d_model]")
        N, F, dm = w_in.shape
        dev = w_in.device
        e4m3 = w_in.dtype == torch.float8_e4m3fn
        if e4m3 != (w_in_scale is not None) or e4m3 != (w_out_scale is not None):
            raise ValueError("float8_e4m3fn experts, and they only, have w_in_scale and w_out_scale")
        self._w_r, self._w_in, self._w_out, self._logit_bias = w_r, w_in, w_out, logit_bias
        self._w_in_scale, self._w_out_scale = w_in_scale, w_out_scale
        self._num_experts, self._d_ff, self._d_model, self._device, self._dtype = N, F, dm, dev, w_in.dtype
        if not e4m3 and w_in.dtype not in (torch.float32, torch.bfloat16):
            raise TypeError(f"w_in must be float32, bfloat16 or float8_e4m3fn, got {w_in.dtype}")
        self._held, self._memory = self._weights(), None
        if capacity is not None and capacity_factor is not None:
            raise ValueError("give capacity or capacity_factor, not both")
        self._top_k, self._capacity, self._capacity_factor, self._flags = int(top_k), capacity, capacity_factor, int(flags)
        self._x_types = {False: (torch.bfloat16,) if e4m3 else (w_in.dtype,), True: (torch.float8_e4m3fn,)}
        self._sizes = {}  # at most 65 entries: more tokens are refused
        self._dims(1)  # refuses sizes that no call could run with

    def _weights(self):
        """Checks the tensors; returns their addresses, in the C function's order."""
        import torch
        N, F, dm, dev, f32 = self._num_experts, self._d_ff, self._d_model, self._device, (torch.float32,)
        return (_want("w_r", self._w_r, (N, dm), f32, dev),
                _want("logit_bias", self._logit_bias, (N,), f32, dev),
                _want("w_in", self._w_in, (N, F, dm), (self._dtype,), dev),
                _want("w_in_scale", self._w_in_scale, (N, F), f32, dev),
                _want("w_out", self._w_out, (N, dm, F), (self._dtype,), dev),
                _want("w_out_scale", self._w_out_scale, (N, dm), f32, dev))

    def _dims(self, T):
        """(dims, their address, workspace bytes) of calls with T tokens."""
        got = self._sizes.get(T)
        if got is None:
            if self._capacity is not None:
                C = int(self._capacity)
            elif self._capacity_factor is not None:
                C = _resolve_capacity(T, self._num_experts, None, self._capacity_factor)
            else:
                C = max(1, T)
            d = dims(T, self._d_model, self._d_ff, self._num_experts, C, _code(self._dtype), self._flags)
            got = self._sizes[T] = (d, ctypes.byref(d), switch_few_workspace_size(d, self._top_k))
        return got

    def __call__(self, x, x_scale=None, out=None, ws=None, stream=None):
        """x [T, d] of the experts' type (8-bit experts: bfloat16, or float8_e4m3fn with x_scale [T] float32).
        Returns a dict with y [T, d] float32 (no residual), aux, expert / gate / slot ([T], or [T, 2] with top_k 2)
        and counts.  ``out`` takes the result of an earlier call with as many tokens, which is overwritten: no input may
        be a part of it."""
        dev = self._device
        if stream is not None:
            with _under(stream, dev):
                return self(x, x_scale, out, ws)
        bias, si, so = self._logit_bias, self._w_in_scale, self._w_out_scale
        held = (self._w_r.data_ptr(), None if bias is None else bias.data_ptr(), self._w_in.data_ptr(),
                None if si is None else si.data_ptr(), self._w_out.data_ptr(), None if so is None else so.data_ptr())
        if held != self._held or self._memory is None:
            # A tensor has other memory than it had: its .data may have been replaced, by something of another size
            # or type too.  The memory is kept, so that nothing else can come to lie at its address unseen.
            self._held = held = self._weights()
            self._memory = [t.detach() for t in (self._w_r, bias, self._w_in, si, self._w_out, so) if t is not None]
        return self._run(x, x_scale, held, out, ws)

    def _run(self, x, x_scale, held, out, ws):
        dev, z = self._device, _names or _torch_names()
        shape, k = x.shape, self._top_k
        if len(shape) != 2:
            raise ValueError(f"x must be [T, {self._d_model}], got {list(shape)}")
        T = shape[0]
        if x_scale is not None and self._w_in_scale is None:
            raise ValueError("x_scale goes with float8_e4m3fn experts and x")
        px = _want("x", x, (T, self._d_model), self._x_types[x_scale is not None], dev)
        pxs = _want("x_scale", x_scale, (T,), z.f32, dev)
        got = self._sizes.get(T)
        d, ref, size = self._dims(T) if got is None else got
        empty, reuse = z.torch.empty, out is not None

        def make():
            pairs, f32, i32 = (T,) if k == 1 else (T, k), z.torch.float32, z.torch.int32
            return dict(y=empty(T, self._d_model, dtype=f32, device=dev), expert=empty(pairs, dtype=i32, device=dev),
                        gate=empty(pairs, dtype=f32, device=dev), slot=empty(pairs, dtype=i32, device=dev),
                        counts=empty(self._num_experts, dtype=i32, device=dev), aux=empty(1, dtype=f32, device=dev))

        out = _result(out, ("few", T, k, self._d_model, self._num_experts, dev), make)
        own = out.own
        if reuse and out.holds(px, pxs):
            out.refuse(x=px, x_scale=pxs)
        if ws is None:
            ws = empty(size, dtype=z.torch.uint8, device=dev)
        else:
            size = ws.numel() * ws.element_size()
            if ws.device != dev:
                raise ValueError(f"ws must be on {dev}, got {ws.device}")
        _launch(lib().switch_layer_fwd_few, "switch_layer_fwd_few", dev, ref, k, px, pxs, *held,
                own["y"].data_ptr(), own["expert"].data_ptr(), own["gate"].data_ptr(), own["slot"].data_ptr(),
                own["counts"].data_ptr(), own["aux"].data_ptr(), _ptr(ws), size)
        out["capacity"], out["flags"], out["workspace"] = d.capacity, d.flags, ws
        return out


for _name in ("w_r", "w_in", "w_out", "logit_bias", "w_in_scale", "w_out_scale", "top_k", "capacity",
              "capacity_factor", "flags", "num_experts", "d_ff", "d_model", "device", "dtype"):
    setattr(FewLayer, _name, property(operator.attrgetter("_" + _name)))
del _name


def layer_fwd_few(x, w_r, w_in, w_out, top_k: int = 1, capacity=None, capacity_factor=None, logit_bias=None,
                  x_scale=None, w_in_scale=None, w_out_scale=None, flags: int = 0, ws=None, out=None, stream=None):
    """layer_fwd / layer_fwd_top2 for up to 64 tokens (see FewLayer, which saves the checks of the weights)."""
    layer = FewLayer(w_r, w_in, w_out, top_k, capacity, capacity_factor, logit_bias, w_in_scale, w_out_scale, flags)
    if stream is not None:
        return layer(x, x_scale, out, ws, stream)
    return layer._run(x, x_scale, layer._held, out, ws)


def block_fwd(residual, norm_weight, w_r, w_in, w_out, delta=None, eps: float = 1e-6, top_k: int = 1, capacity=None,
              capacity_factor=None, logit_bias=None, w_in_scale=None, w_out_scale=None, flags: int = 0, stream=None):
    """One pre-norm block: s = residual + delta, x = s / rms(s) * norm_weight, y = layer(x); the caller adds y as
    the next block's delta.  Up to 64 tokens outside of training go through switch_layer_fwd_few (8-bit experts
    always do, with x in 8 bits: more tokens are refused), others through switch_layer_fwd / switch_layer_fwd_top2.
    Sizes and options that the layer for few tokens cannot run with are refused before the norm is launched.  Returns
    the layer's dict with sum (residual where there is no delta), x, x_scale and rstd besides."""
    import torch
    if stream is not None:
        with _under(stream, residual.device):
            return block_fwd(residual, norm_weight, w_r, w_in, w_out, delta, eps, top_k, capacity, capacity_factor,
                             logit_bias, w_in_scale, w_out_scale, flags)
    T, e4m3 = residual.shape[0], w_in.dtype == torch.float8_e4m3fn
    if top_k not in (1, 2):
        raise ValueError("top_k must be 1 or 2")
    if capacity is None and capacity_factor is None:
        raise ValueError("give capacity or capacity_factor")
    if e4m3 and T > SWITCH_FEW_MAX_TOKENS:
        raise ValueError(f"float8_e4m3fn experts take at most {SWITCH_FEW_MAX_TOKENS} tokens, got {T}")
    layer = None
    if e4m3 or (T <= SWITCH_FEW_MAX_TOKENS and (flags & ~SWITCH_FLAG_SIMT_FFN) == 0):
        layer = FewLayer(w_r, w_in, w_out, top_k, capacity, capacity_factor, logit_bias, w_in_scale, w_out_scale, flags)
    n = norm_fwd(residual, norm_weight, delta=delta, eps=eps, out_dtype=w_in.dtype)
    x = n["out"]
    if layer is not None:
        r = layer._run(x, n["scale"], layer._held, None, None)
    else:
        with _current(x.device):
            r = (layer_fwd if top_k == 1 else layer_fwd_top2)(x, w_r, w_in, w_out, capacity, capacity_factor,
                                                              logit_bias, flags)
    return dict(r, sum=residual if delta is None else n["sum"], x=x, x_scale=n["scale"], rstd=n["rstd"])


def block_bwd(fwd: dict, norm_weight, w_r, w_in, w_out, dy, dsum=None, g_aux: float = 0.0, logit_bias=None,
              stream=None):
    """Gradients of sum(y * dy) + sum(s * dsum) + g_aux * aux after ``block_fwd(..., flags=SWITCH_FLAG_TRAINING)`` with
    top_k 1 (the top-2 layer has no backward pass, and is refused):
    layer_bwd's dw_r, dbias, dw_in, dw_out, with dresidual (of residual and delta alike) and dnorm_weight, float32."""
    if stream is not None:
        with _under(stream, dy.device):  # dx, which dies here, is allocated on the stream that it is used on
            return block_bwd(fwd, norm_weight, w_r, w_in, w_out, dy, dsum, g_aux, logit_bias)
    with _current(dy.device):
        g = layer_bwd(fwd, fwd["x"], w_r, w_in, w_out, dy, g_aux, logit_bias)
    n = norm_bwd(fwd["sum"], norm_weight, fwd["rstd"], g.pop("dx"), dsum=dsum)
    return dict(g, dresidual=n["dresidual"], dnorm_weight=n["dweight"])
