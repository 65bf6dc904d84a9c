"""SmoothQuant W8A8 INT8 linear layer for NVIDIA B200 (sm_100a).

Thin Python binding over libsq (the C ABI in include/sq.h).  Every function
here only marshals arguments -- tensors become device pointers, the current
torch CUDA stream becomes the stream argument -- and raises ``SQError`` when
the library returns an error.  All arithmetic runs in the library's CUDA
kernels; there is no CPU fallback: if libsq.so cannot be loaded, every call
raises.

The raw entry points keep the C names and take caller-allocated outputs:

    sq_calib_absmax(x, ax)                      ax[K] accumulated by max
    sq_smooth_factors(ax, w, alpha, s, aw=None)
    sq_smooth_quant_weight(w, s, wq, sw)
    sq_quant_act(x, s, xq, sx)
    sq_w8a8_gemm(xq, sx, wq, sw, y)
    sq_w8a8_gemm_ws(xq, sx, wq, sw, y, workspace)   every SM busy whatever the shape
    sq_w8a8_gemm_workspace_size(M, N, K)
    sq_w8a8_gemm_s32(xq, wq, acc)
    sq_linear(x, s, wq, sw, y, workspace)
    sq_linear_workspace_size(M, N, K)
    sq_linear_noalloc(x, s, wq, sw, y)          no workspace, no allocation
    sq_mx4_quant_act(x, s, xq, sx)              microscaled 4-bit (MXFP4): codes and scale tiles
    sq_mx4_quant_weight(w, s, wq, sw)
    sq_mx4_dequant(q, sc, out)
    sq_mx4_gemm(xq, sx, wq, sw, y, workspace)
    sq_mx4_linear(x, s, wq, sw, y, workspace)
    sq_mx4_moe(xq, sx, ids, weights, wg, sg, wu, su, wd, sd, y, workspace)   a few tokens through their experts
    sq_residual_norm_quant(b, gamma, gate, gate_tokens, c, r, r_out, g, eps, xq, sx)   norms around a block, int8 out
    sq_residual_norm_quant_mx4(...)             the same, MXFP4 out
    sq_device_status()

``calibrate``, ``prepare_weight`` and ``linear`` are conveniences that allocate
their outputs with torch and call the raw entry points.

With ``stream=`` (a torch stream or a raw handle) a call runs there instead of on
the current stream, and what it allocates, workspaces and outputs, belongs to
that stream: wait for it before an output is used on another one.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading
from typing import Optional, Tuple

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsq.so")

SQ_OK, SQ_ERR_INVALID_ARG, SQ_ERR_UNSUPPORTED, SQ_ERR_CUDA, SQ_ERR_TIMEOUT = range(5)
SQ_F32, SQ_BF16 = 0, 1

# every symbol include/sq.h declares
ABI_SYMBOLS = (
    "sq_status_string",
    "sq_version",
    "sq_calib_absmax",
    "sq_smooth_factors",
    "sq_smooth_quant_weight",
    "sq_quant_act",
    "sq_fold_gamma",
    "sq_rmsnorm_quant",
    "sq_silu_mul_quant",
    "sq_gptq_workspace_size",
    "sq_gptq_hessian",
    "sq_gptq_factor",
    "sq_gptq_quant_weight",
    "sq_w8a8_gemm",
    "sq_w8a8_gemm_ws",
    "sq_w8a8_gemm_workspace_size",
    "sq_w8a8_gemm_s32",
    "sq_linear",
    "sq_linear_workspace_size",
    "sq_linear_noalloc",
    "sq_mx4_scale_size",
    "sq_mx4_quant_act",
    "sq_mx4_quant_weight",
    "sq_mx4_dequant",
    "sq_mx4_gemm_workspace_size",
    "sq_mx4_gemm",
    "sq_mx4_linear_workspace_size",
    "sq_mx4_linear",
    "sq_mx4_moe_workspace_size",
    "sq_mx4_moe",
    "sq_residual_norm_quant",
    "sq_residual_norm_quant_mx4",
    "sq_device_status",
    "sq_selftest_wait_timeout",
)


class SQError(RuntimeError):
    def __init__(self, fn: str, status: int, name: str):
        super().__init__(f"{fn} failed: {name} ({status})")
        self.status = status
        self.fn = fn


_lock = threading.Lock()
_lib = None


def _declare(lib):
    P, I, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float
    E, Z = ctypes.c_int, ctypes.c_size_t
    sig = {
        "sq_status_string": ([E], ctypes.c_char_p),
        "sq_version": ([], ctypes.c_int),
        "sq_calib_absmax": ([P, E, I, I, I, P, P], E),
        "sq_smooth_factors": ([P, P, E, I, I, F, P, P, P], E),
        "sq_smooth_quant_weight": ([P, E, I, I, P, P, P, P], E),
        "sq_quant_act": ([P, E, I, I, P, P, P, P], E),
        "sq_fold_gamma": ([P, P, I, P, P], E),
        "sq_rmsnorm_quant": ([P, E, I, I, P, F, P, P, P, P], E),
        "sq_silu_mul_quant": ([P, E, I, I, P, P, P, P, P], E),
        "sq_gptq_workspace_size": ([I], ctypes.c_size_t),
        "sq_gptq_hessian": ([P, E, I, I, P, P, P], E),
        "sq_gptq_factor": ([P, I, F, P, P, ctypes.c_size_t, P], E),
        "sq_gptq_quant_weight": ([P, E, I, I, P, P, P, P, P], E),
        "sq_w8a8_gemm": ([P, P, P, P, I, I, I, P, E, P], E),
        "sq_w8a8_gemm_ws": ([P, P, P, P, I, I, I, P, E, P, ctypes.c_size_t, P], E),
        "sq_w8a8_gemm_workspace_size": ([I, I, I], ctypes.c_size_t),
        "sq_w8a8_gemm_s32": ([P, P, I, I, I, P, P], E),
        "sq_linear": ([P, E, P, P, P, I, I, I, P, E, P, ctypes.c_size_t, P], E),
        "sq_linear_workspace_size": ([I, I, I], ctypes.c_size_t),
        "sq_linear_noalloc": ([P, E, P, P, P, I, I, I, P, E, P], E),
        "sq_mx4_scale_size": ([I, I], Z),
        "sq_mx4_quant_act": ([P, E, I, I, P, P, P, P], E),
        "sq_mx4_quant_weight": ([P, E, I, I, P, P, P, P], E),
        "sq_mx4_dequant": ([P, P, I, I, P, E, P], E),
        "sq_mx4_gemm_workspace_size": ([I, I, I], Z),
        "sq_mx4_gemm": ([P, P, P, P, I, I, I, P, E, P, Z, P], E),
        "sq_mx4_linear_workspace_size": ([I, I, I], Z),
        "sq_mx4_linear": ([P, E, P, P, P, I, I, I, P, E, P, Z, P], E),
        "sq_mx4_moe_workspace_size": ([I, I, I, I, I], Z),
        "sq_mx4_moe": ([P, P, P, P, I, I, I, I, I, P, P, P, P, P, P, P, E, P, Z, P], E),
        "sq_residual_norm_quant": ([P, E, I, I, P, P, I, F, P, P, P, F, P, P, P], E),
        "sq_residual_norm_quant_mx4": ([P, E, I, I, P, P, I, F, P, P, P, F, P, P, P], E),
        "sq_device_status": ([P, ctypes.POINTER(ctypes.c_uint32)], E),
        "sq_selftest_wait_timeout": ([ctypes.c_uint32, P], E),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res


def lib():
    """The loaded libsq (ctypes.CDLL).  Raises if the library is not built."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise ImportError(
                    f"libsq.so is not built at {LIB_PATH}; run "
                    "`python -m w8a8_int8_gemm_channel_b200._build` (needs nvcc)"
                )
            l = ctypes.CDLL(LIB_PATH)
            _declare(l)
            _lib = l
    return _lib


def status_string(st: int) -> str:
    return lib().sq_status_string(st).decode()


def _check(fn: str, st: int):
    if st != SQ_OK:
        raise SQError(fn, st, status_string(st))


def _torch():
    import torch

    return torch


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return SQ_F32
    if t.dtype == torch.bfloat16:
        return SQ_BF16
    raise TypeError(f"unsupported dtype {t.dtype}; expected float32 or bfloat16")


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libsq takes device tensors")
    if not t.is_contiguous():
        raise ValueError("libsq takes contiguous tensors")
    return t.data_ptr()


def _stream(stream=None) -> int:
    torch = _torch()
    if stream is None:
        # the raw handle, where torch gives it: a Stream object costs more than a launch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:
            return raw(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


_HERE = contextlib.nullcontext()


def _on(stream, device):
    """Context in which torch allocates and fills on the stream that a call is launched on.  A tensor allocated on the
    current stream may be written there by earlier work, and is given to later work there as soon as it is dropped: both
    while `stream` uses it."""
    if stream is None:
        return _HERE
    torch = _torch()
    if not hasattr(stream, "cuda_stream"):
        handle = int(stream)  # 0 and 1 name the legacy default stream
        stream = torch.cuda.ExternalStream(handle, device=device) if handle > 1 else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def _scratch(nbytes: int, device, stream):
    torch = _torch()
    with _on(stream, device):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


# ---------------------------------------------------------------------------
# raw entry points (C names)
# ---------------------------------------------------------------------------

def sq_calib_absmax(x, ax, stream=None):
    T, K = x.shape
    _check("sq_calib_absmax",
           lib().sq_calib_absmax(_ptr(x), _dtype_code(x), T, K, K, _ptr(ax), _stream(stream)))


def sq_smooth_factors(ax, w, alpha: float, s, aw=None, stream=None):
    N, K = w.shape
    _check("sq_smooth_factors",
           lib().sq_smooth_factors(_ptr(ax), _ptr(w), _dtype_code(w), N, K, float(alpha), _ptr(s),
                                   _ptr(aw), _stream(stream)))


def sq_smooth_quant_weight(w, s, wq, sw, stream=None):
    N, K = w.shape
    _check("sq_smooth_quant_weight",
           lib().sq_smooth_quant_weight(_ptr(w), _dtype_code(w), N, K, _ptr(s), _ptr(wq), _ptr(sw),
                                        _stream(stream)))


def sq_quant_act(x, s, xq, sx, stream=None):
    M, K = x.shape
    _check("sq_quant_act",
           lib().sq_quant_act(_ptr(x), _dtype_code(x), M, K, _ptr(s), _ptr(xq), _ptr(sx),
                              _stream(stream)))


def sq_fold_gamma(gamma, s, g, stream=None):
    K = gamma.shape[0]
    _check("sq_fold_gamma", lib().sq_fold_gamma(_ptr(gamma), _ptr(s), K, _ptr(g), _stream(stream)))


def sq_rmsnorm_quant(h, g, eps, xq, sx, rinv=None, stream=None):
    M, K = h.shape
    _check("sq_rmsnorm_quant",
           lib().sq_rmsnorm_quant(_ptr(h), _dtype_code(h), M, K, _ptr(g), float(eps), _ptr(xq), _ptr(sx),
                                  None if rinv is None else _ptr(rinv), _stream(stream)))


def sq_silu_mul_quant(gu, s, xq, sx, h=None, stream=None):
    """gu [M, 2I] = [gate | up] rows; xq [M, I] int8 and sx [M] fp32 out; h [M, I]
    (gu's dtype) receives SiLU(gate) * up when given."""
    M, I2 = gu.shape
    _check("sq_silu_mul_quant",
           lib().sq_silu_mul_quant(_ptr(gu), _dtype_code(gu), M, I2 // 2, _ptr(s), _ptr(xq), _ptr(sx),
                                   None if h is None else _ptr(h), _stream(stream)))


def sq_gptq_hessian(x, s, H, stream=None):
    """H [K, K] fp64 = xh^T xh over the calibration tokens x [T, K] (xh = x / s)."""
    T, K = x.shape
    _check("sq_gptq_hessian", lib().sq_gptq_hessian(_ptr(x), _dtype_code(x), T, K, _ptr(s), _ptr(H), _stream(stream)))


def sq_gptq_factor(H, U, damp_frac=0.01, workspace=None, stream=None):
    """Damps H in place and writes U, the upper Cholesky factor of H^-1."""
    K = H.shape[0]
    need = int(lib().sq_gptq_workspace_size(K))
    if workspace is None:
        workspace = _scratch(need, H.device, stream)
    _check("sq_gptq_factor", lib().sq_gptq_factor(_ptr(H), K, float(damp_frac), _ptr(U), _ptr(workspace),
                                                  workspace.numel() * workspace.element_size(), _stream(stream)))


def sq_gptq_quant_weight(w, s, U, wq, sw, stream=None):
    """GPTQ codes wq [N, K] and per-channel scales sw [N] of the smoothed weight."""
    N, K = w.shape
    _check("sq_gptq_quant_weight", lib().sq_gptq_quant_weight(_ptr(w), _dtype_code(w), N, K, _ptr(s), _ptr(U),
                                                              _ptr(wq), _ptr(sw), _stream(stream)))


def gptq_weight(xcal, w, s, damp_frac=0.01, stream=None):
    """GPTQ in place of prepare_weight's plain rounding: (wq, sw) for the
    smoothed weight w * s, with the Hessian from the calibration tokens xcal."""
    torch = _torch()
    K = w.shape[1]
    with _on(stream, w.device):
        H = torch.empty(K, K, dtype=torch.float64, device=w.device)
        U = torch.empty_like(H)
        sq_gptq_hessian(xcal, s, H, stream)
        sq_gptq_factor(H, U, damp_frac, stream=stream)
        wq = torch.empty(w.shape, dtype=torch.int8, device=w.device)
        sw = torch.empty(w.shape[0], dtype=torch.float32, device=w.device)
        sq_gptq_quant_weight(w, s, U, wq, sw, stream)
    return wq, sw


def sq_w8a8_gemm(xq, sx, wq, sw, y, stream=None):
    M, K = xq.shape
    N = wq.shape[0]
    _check("sq_w8a8_gemm",
           lib().sq_w8a8_gemm(_ptr(xq), _ptr(sx), _ptr(wq), _ptr(sw), M, N, K, _ptr(y),
                              _dtype_code(y), _stream(stream)))


def sq_w8a8_gemm_workspace_size(M: int, N: int, K: int) -> int:
    return int(lib().sq_w8a8_gemm_workspace_size(M, N, K))


def sq_w8a8_gemm_ws(xq, sx, wq, sw, y, workspace=None, stream=None):
    """sq_w8a8_gemm with a workspace (allocated here when not given)."""
    M, K = xq.shape
    N = wq.shape[0]
    if workspace is None:
        workspace = _scratch(sq_w8a8_gemm_workspace_size(M, N, K), xq.device, stream)
    _check("sq_w8a8_gemm_ws",
           lib().sq_w8a8_gemm_ws(_ptr(xq), _ptr(sx), _ptr(wq), _ptr(sw), M, N, K, _ptr(y), _dtype_code(y),
                                 _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def sq_w8a8_gemm_s32(xq, wq, acc, stream=None):
    M, K = xq.shape
    N = wq.shape[0]
    _check("sq_w8a8_gemm_s32",
           lib().sq_w8a8_gemm_s32(_ptr(xq), _ptr(wq), M, N, K, _ptr(acc), _stream(stream)))


def sq_linear_workspace_size(M: int, N: int, K: int) -> int:
    return int(lib().sq_linear_workspace_size(M, N, K))


def sq_linear(x, s, wq, sw, y, workspace=None, stream=None):
    M, K = x.shape
    N = wq.shape[0]
    ws_ptr = None if workspace is None else _ptr(workspace)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("sq_linear",
           lib().sq_linear(_ptr(x), _dtype_code(x), _ptr(s), _ptr(wq), _ptr(sw), M, N, K, _ptr(y),
                           _dtype_code(y), ws_ptr, ws_bytes, _stream(stream)))


# bytes of the library's fixed scratch array used by sq_linear_noalloc
LINEAR_NOALLOC_SCRATCH_BYTES = 32 << 20


def sq_linear_noalloc(x, s, wq, sw, y, stream=None):
    """sq_linear with the library's own fixed scratch array instead of a
    caller workspace; allocates nothing.  Raises SQError(SQ_ERR_UNSUPPORTED)
    when sq_linear_workspace_size(M, N, K) exceeds
    LINEAR_NOALLOC_SCRATCH_BYTES."""
    M, K = x.shape
    N = wq.shape[0]
    _check("sq_linear_noalloc",
           lib().sq_linear_noalloc(_ptr(x), _dtype_code(x), _ptr(s), _ptr(wq), _ptr(sw), M, N, K,
                                   _ptr(y), _dtype_code(y), _stream(stream)))


# ---------------------------------------------------------------------------
# microscaled 4-bit (MXFP4): s may be None; codes are uint8 [rows, K / 2], scales
# uint8 of sq_mx4_scale_size(rows, K) bytes in the tiles include/sq.h describes
# ---------------------------------------------------------------------------

def _need(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


_codes_of = {}  # torch dtype -> code of the mx4 calls, and what else of torch they use (filled once it is imported)


def _torch_parts():
    """(uint8, float32, current device's number, current stream's raw handle of a device)."""
    parts = _codes_of.get("parts")
    if parts is None:
        torch = _torch()
        _codes_of[torch.float32], _codes_of[torch.bfloat16] = SQ_F32, SQ_BF16
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda d: torch.cuda.current_stream(d).cuda_stream)
        device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        parts = _codes_of["parts"] = (torch.uint8, torch.float32, device, raw)
    return parts


def _code(t) -> int:
    c = _codes_of.get(t.dtype)
    if c is None:
        raise TypeError(f"unsupported dtype {t.dtype}; expected float32 or bfloat16")
    return c


def _mx4_ptrs(rows: int, K: int, q, sc):
    """Device pointers of codes and scales, their sizes checked against [rows, K]."""
    u8 = _torch_parts()[0]
    if q.dtype is not u8 or q.shape != (rows, K // 2):
        raise ValueError(f"codes: uint8 of shape {(rows, K // 2)}")
    if sc.dtype is not u8 or sc.numel() < ((rows + 127) >> 7) * ((K + 127) >> 7) * 512:
        raise ValueError(f"scales: uint8 of sq_mx4_scale_size({rows}, {K}) bytes")
    return q.data_ptr(), sc.data_ptr()


def _mx4_factors(s, K: int):
    if s is None:
        return None
    if s.dtype is not _torch_parts()[1] or s.numel() != K:
        raise ValueError(f"s: float32 of {K} values")
    return s.data_ptr()


def _ws_args(ws):
    return (None, 0) if ws is None else (ws.data_ptr(), ws.numel() * ws.element_size())


def _call(name, stream, tensors, make_args):
    """Calls an entry point with the tensors' device current: every tensor on one device and contiguous (None: left
    out).  make_args() gives the arguments before the stream."""
    _, _, device, raw_stream = _torch_parts()
    d = tensors[0].get_device()
    for t in tensors:
        if t is not None and (t.get_device() != d or d < 0 or not t.is_contiguous()):
            if not t.is_cuda:
                raise ValueError("libsq takes device tensors")
            raise ValueError("libsq takes contiguous tensors" if t.get_device() == d else f"tensors on devices {d} and {t.get_device()}")
    f = getattr(_lib or lib(), name)
    if d == device():
        st = f(*make_args(), raw_stream(d) if stream is None else _stream(stream))
    else:
        with _torch().cuda.device(d):
            st = f(*make_args(), raw_stream(d) if stream is None else _stream(stream))
    if st != SQ_OK:
        raise SQError(name, st, status_string(st))


def sq_mx4_scale_size(rows: int, K: int) -> int:
    """Bytes of the scale tiles of a [rows, K] matrix."""
    return int(lib().sq_mx4_scale_size(rows, K))


def sq_mx4_quant_act(x, s, xq, sx, stream=None):
    M, K = x.shape
    _call("sq_mx4_quant_act", stream, (x, s, xq, sx),
          lambda: (x.data_ptr(), _code(x), M, K, _mx4_factors(s, K), *_mx4_ptrs(M, K, xq, sx)))


def sq_mx4_quant_weight(w, s, wq, sw, stream=None):
    N, K = w.shape
    _call("sq_mx4_quant_weight", stream, (w, s, wq, sw),
          lambda: (w.data_ptr(), _code(w), N, K, _mx4_factors(s, K), *_mx4_ptrs(N, K, wq, sw)))


def sq_mx4_dequant(q, sc, out, stream=None):
    """out [rows, K] (float32 or bfloat16): the values the codes stand for."""
    rows, K = out.shape
    _call("sq_mx4_dequant", stream, (out, q, sc),
          lambda: (*_mx4_ptrs(rows, K, q, sc), rows, K, out.data_ptr(), _code(out)))


def sq_mx4_gemm_workspace_size(M: int, N: int, K: int) -> int:
    return int(lib().sq_mx4_gemm_workspace_size(M, N, K))


def sq_mx4_gemm(xq, sx, wq, sw, y, workspace=None, stream=None):
    """y [M, N] = x w^T of the values the codes stand for (a workspace is allocated when none is given)."""
    M, N = y.shape
    K = xq.shape[1] * 2
    if workspace is None:
        workspace = _scratch(sq_mx4_gemm_workspace_size(M, N, K), y.device, stream)
    _call("sq_mx4_gemm", stream, (y, xq, sx, wq, sw, workspace),
          lambda: (*_mx4_ptrs(M, K, xq, sx), *_mx4_ptrs(N, K, wq, sw), M, N, K, y.data_ptr(), _code(y),
                   *_ws_args(workspace)))


def sq_mx4_linear_workspace_size(M: int, N: int, K: int) -> int:
    return int(lib().sq_mx4_linear_workspace_size(M, N, K))


def sq_mx4_linear(x, s, wq, sw, y, workspace=None, stream=None):
    """y [M, N] = mx4(x * (1 / s)) w^T (a workspace is allocated when none is given)."""
    M, K = x.shape
    N = wq.shape[0]
    if y.shape != (M, N):
        raise ValueError(f"y: shape {(M, N)}")
    if workspace is None:
        workspace = _scratch(sq_mx4_linear_workspace_size(M, N, K), x.device, stream)
    _call("sq_mx4_linear", stream, (x, s, wq, sw, y, workspace),
          lambda: (x.data_ptr(), _code(x), _mx4_factors(s, K), *_mx4_ptrs(N, K, wq, sw), M, N, K, y.data_ptr(),
                   _code(y), *_ws_args(workspace)))


def sq_mx4_moe_workspace_size(T: int, topk: int, E: int, H: int, I: int) -> int:
    return int(lib().sq_mx4_moe_workspace_size(T, topk, E, H, I))


def sq_mx4_moe(xq, sx, ids, weights, wg, sg, wu, su, wd, sd, y, workspace=None, stream=None):
    """y [T, H] = the weighted sum over each token's experts ids [T, topk] (int32; outside [0, E): none) of the gated
    layer wd[e] (silu(wg[e] x) * (wu[e] x)); x as codes xq [T, H / 2] and scale tiles sx."""
    torch = _torch()
    T, topk = ids.shape
    E, I, H2 = wg.shape
    H, u8 = H2 * 2, torch.uint8
    if ids.dtype is not torch.int32 or weights.dtype is not torch.float32 or weights.shape != (T, topk):
        raise ValueError("ids: int32, weights: float32, both [T, topk]")
    if wu.shape != (E, I, H2) or wd.shape != (E, H, I // 2) or not (wg.dtype is wu.dtype is wd.dtype is u8):
        raise ValueError("wg, wu: uint8 [E, I, H / 2], wd: uint8 [E, H, I / 2]")
    kt_h, kt_i = -(-H // 128), -(-I // 128)
    size = (E, kt_i * kt_h * 512)
    if sg.shape != size or su.shape != size or sd.shape != size or not (sg.dtype is su.dtype is sd.dtype is u8):
        raise ValueError(f"scales: uint8 {size}")
    if y.shape != (T, H):
        raise ValueError(f"y: shape {(T, H)}")
    if workspace is None:
        workspace = _scratch(sq_mx4_moe_workspace_size(T, topk, E, H, I), y.device, stream)
    _call("sq_mx4_moe", stream, (y, xq, sx, ids, weights, wg, sg, wu, su, wd, sd, workspace),
          lambda: (*_mx4_ptrs(T, H, xq, sx), ids.data_ptr(), weights.data_ptr(), T, topk, E, H, I, wg.data_ptr(),
                   sg.data_ptr(), wu.data_ptr(), su.data_ptr(), wd.data_ptr(), sd.data_ptr(), y.data_ptr(),
                   _code(y), *_ws_args(workspace)))


def _residual_norm(name, b, gamma, gate, gate_tokens, c, r, r_out, g, eps, q, sx, stream):
    M, K = b.shape
    if r.shape != b.shape or r_out.shape != b.shape or not (b.dtype is r.dtype is r_out.dtype):
        raise ValueError(f"b, r and r_out: shape {(M, K)} and one dtype")
    if gate is not None and (gate_tokens < 1 or gate.dtype is not b.dtype or gate.shape[-1] != K or
                             gate.numel() < -(-M // gate_tokens) * K):
        raise ValueError("gate: b's dtype, a row for every gate_tokens tokens")
    _call(name, stream, (b, gamma, gate, r, r_out, g, q, sx),
          lambda: (b.data_ptr(), _code(b), M, K, _mx4_factors(gamma, K), None if gate is None else gate.data_ptr(),
                   int(gate_tokens), float(c), r.data_ptr(), r_out.data_ptr(), _mx4_factors(g, K), float(eps),
                   q.data_ptr(), sx.data_ptr()))


def sq_residual_norm_quant(b, gamma, gate, gate_tokens, c, r, r_out, g, eps, xq, sx, stream=None):
    """r_out = r + c * gate * rmsnorm(b, gamma) (gamma, gate: None to leave out; r_out may be r); xq [M, K] int8 and
    sx [M]: rmsnorm(r_out, g) quantised per token.  Token m uses gate row m // gate_tokens."""
    _need(xq.dtype is _torch().int8 and xq.shape == b.shape, f"xq: int8 of shape {tuple(b.shape)}")
    _need(sx.dtype is _torch().float32 and sx.numel() == b.shape[0], f"sx: float32 of {b.shape[0]} values")
    _residual_norm("sq_residual_norm_quant", b, gamma, gate, gate_tokens, c, r, r_out, g, eps, xq, sx, stream)


def sq_residual_norm_quant_mx4(b, gamma, gate, gate_tokens, c, r, r_out, g, eps, xq, sx, stream=None):
    """sq_residual_norm_quant with MXFP4 codes xq [M, K / 2] and scale tiles sx."""
    _mx4_ptrs(*b.shape, xq, sx)
    _residual_norm("sq_residual_norm_quant_mx4", b, gamma, gate, gate_tokens, c, r, r_out, g, eps, xq, sx, stream)


def sq_device_status(stream=None) -> Tuple[int, int]:
    code = ctypes.c_uint32(0)
    st = lib().sq_device_status(_stream(stream), ctypes.byref(code))
    return st, int(code.value)


def sq_selftest_wait_timeout(limit_us: int, stream=None):
    _check("sq_selftest_wait_timeout", lib().sq_selftest_wait_timeout(int(limit_us), _stream(stream)))


# ---------------------------------------------------------------------------
# conveniences (allocate outputs with torch, then call the raw entry points)
# ---------------------------------------------------------------------------

def calibrate(x_batches, K: Optional[int] = None, stream=None):
    """Accumulate the per-channel absmax A_j over one or more calibration batches."""
    torch = _torch()
    batches = [x_batches] if hasattr(x_batches, "shape") else list(x_batches)
    K = K or batches[0].shape[1]
    with _on(stream, batches[0].device):
        ax = torch.zeros(K, dtype=torch.float32, device=batches[0].device)
        for b in batches:
            sq_calib_absmax(b, ax, stream)
    return ax


def prepare_weight(ax, w, alpha: float, stream=None):
    """Smoothing factors and the smoothed int8 weight: returns (s, wq, sw)."""
    torch = _torch()
    N, K = w.shape
    with _on(stream, w.device):
        s = torch.empty(K, dtype=torch.float32, device=w.device)
        sq_smooth_factors(ax, w, alpha, s, None, stream)
        wq = torch.empty(N, K, dtype=torch.int8, device=w.device)
        sw = torch.empty(N, dtype=torch.float32, device=w.device)
        sq_smooth_quant_weight(w, s, wq, sw, stream)
    return s, wq, sw


def linear(x, s, wq, sw, out_dtype=None, workspace=None, stream=None):
    """Y = dequant(quant(X / s) @ Wq^T) with a torch-allocated output."""
    torch = _torch()
    M, K = x.shape
    N = wq.shape[0]
    with _on(stream, x.device):
        y = torch.empty(M, N, dtype=out_dtype or x.dtype, device=x.device)
        need = sq_linear_workspace_size(M, N, K)
        if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
            workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
        sq_linear(x, s, wq, sw, y, workspace if need else None, stream)
    return y


def mx4_quantize(x, s=None, stream=None):
    """Codes and scale tiles of the activations x [M, K], times the rounded 1 / s when given: returns (xq, sx)."""
    torch = _torch()
    M, K = x.shape
    with _on(stream, x.device):
        xq = torch.empty(M, K // 2, dtype=torch.uint8, device=x.device)
        sx = torch.empty(sq_mx4_scale_size(M, K), dtype=torch.uint8, device=x.device)
    sq_mx4_quant_act(x, s, xq, sx, stream)
    return xq, sx


def mx4_prepare_weight(w, s=None, stream=None):
    """Codes and scale tiles of a weight [N, K] (times s when given), or of each of the experts' weights [E, N, K]:
    returns (wq, sw), [N, K / 2] and [bytes] or [E, N, K / 2] and [E, bytes]."""
    torch = _torch()
    N, K = w.shape[-2:]
    with _on(stream, w.device):
        wq = torch.empty(*w.shape[:-1], K // 2, dtype=torch.uint8, device=w.device)
        sw = torch.empty(*w.shape[:-2], sq_mx4_scale_size(N, K), dtype=torch.uint8, device=w.device)
    for one, q, sc in zip(*(t.reshape(-1, *t.shape[-d:]) for t, d in ((w, 2), (wq, 2), (sw, 1)))):
        sq_mx4_quant_weight(one, s, q, sc, stream)
    return wq, sw


def mx4_linear(x, s, wq, sw, out_dtype=None, workspace=None, stream=None):
    """y = mx4(x * (1 / s)) w^T with a torch-allocated output."""
    with _on(stream, x.device):
        y = _torch().empty(x.shape[0], wq.shape[0], dtype=out_dtype or x.dtype, device=x.device)
    sq_mx4_linear(x, s, wq, sw, y, workspace, stream)
    return y


def mx4_moe(xq, sx, ids, weights, wg, sg, wu, su, wd, sd, out_dtype=None, workspace=None, stream=None):
    """A few tokens through their experts with a torch-allocated output (bfloat16 unless out_dtype says otherwise)."""
    torch = _torch()
    with _on(stream, xq.device):
        y = torch.empty(ids.shape[0], wd.shape[1], dtype=out_dtype or torch.bfloat16, device=xq.device)
    sq_mx4_moe(xq, sx, ids, weights, wg, sg, wu, su, wd, sd, y, workspace, stream)
    return y
