"""Thin Python binding of libw2a8.so (the MI355X W2A8 linear layer).

Every function marshals arguments (dtype, shape, device, contiguity checks;
pointers and the current HIP stream) and calls the C ABI of the same name in
``include/w2a8.h``; all computation happens in the library.  PyTorch supplies
device memory and streams only.  If the library has not been built, importing
the binding's functions raises; there is no fallback path.

Host functions take/return CPU tensors; device functions take CUDA (HIP)
tensors on the current device and enqueue work on the current stream (or on
``stream=`` if given).
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

__all__ = [
    "W2A8Error", "lib", "packed_bytes", "workspace_bytes", "layout_version",
    "ternarize_absmean", "pack_ternary", "unpack_ternary", "quant_act_int8",
    "w2a8_gemv", "w2a8_gemv_noalloc", "w2a8_gemm", "gemv", "gemm", "linear", "Workspace",
    "w2a8_linear_gemv", "tune_gemv", "tune_gemv_force", "gemv_plan", "linear_plan", "mx4_plan", "DEFAULT_GEMV_POLICY",
    "tune_gemm", "tune_gemm_ring", "tune_gemm_pipe",
    "act4_bytes", "pack_act_int4", "quant_act_int4", "w2a4_gemv", "w2a4_linear_gemv",
    "linear_a4", "w2a8_gemv_grouped", "w2a8_linear_gemv_grouped", "linear_grouped",
    "mx4_act_bytes", "mx4_scale_bytes", "mx4_packed_bytes", "pack_mx4", "unpack_mx4",
    "quant_act_mx4", "dequant_act_mx4", "quant_pack_mx4", "w4mx4_gemm", "w2mx4_gemm",
    "w4mx4_linear_gemv", "w2mx4_linear_gemv", "gemm_w4mx4", "gemm_w2mx4", "linear_w4mx4",
    "linear_w2mx4", "rmsnorm_quant_int8", "w4a8_packed_bytes", "pack_w4a8", "unpack_w4a8",
    "w4a8_workspace_bytes", "w4a8_gemm", "gemm_w4a8", "linear_w4a8", "w2a8_moe_workspace_bytes", "w2a8_moe", "moe",
    "w4a8_plan", "moe_plan", "tune_moe",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libw2a8.so")
LAYOUT_VERSION = 1

_lib = None
_lib_lock = threading.Lock()


class W2A8Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {lib().w2a8_status_str(status).decode()} (status {status})")


def lib():
    """The loaded library (built in-tree); raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    with _lib_lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is not built; run `python -c 'import __graft_entry__ as g; g.build()'` "
                "or `python w2a8_gemv_amd/build.py`")
        L = ctypes.CDLL(LIB_PATH)
        P, I64, I32, F32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
        L.w2a8_status_str.argtypes = [I32]
        L.w2a8_status_str.restype = ctypes.c_char_p
        L.w2a8_layout_version.argtypes = []
        L.w2a8_layout_version.restype = I32
        L.w2a8_packed_bytes.argtypes = [I64, I64]
        L.w2a8_packed_bytes.restype = I64
        L.w2a8_workspace_bytes.argtypes = [I64, I64, I64]
        L.w2a8_workspace_bytes.restype = I64
        L.w2a8_ternarize_absmean.argtypes = [P, I64, I64, P, P]
        L.w2a8_ternarize_absmean.restype = I32
        L.pack_ternary.argtypes = [P, I64, I64, P, I64]
        L.pack_ternary.restype = I32
        L.unpack_ternary.argtypes = [P, I64, I64, I64, P]
        L.unpack_ternary.restype = I32
        L.quant_act_int8.argtypes = [P, I64, I64, P, P, P]
        L.quant_act_int8.restype = I32
        L.w2a8_gemv.argtypes = [P, P, I64, I64, P, P, F32, P, P, I64, P]
        L.w2a8_gemv.restype = I32
        L.w2a8_gemv_noalloc.argtypes = [P, P, I64, I64, P, P, F32, P, P]
        L.w2a8_gemv_noalloc.restype = I32
        L.w2a8_gemm.argtypes = [P, P, I64, I64, I64, P, P, F32, P, P, I64, P]
        L.w2a8_gemm.restype = I32
        L.w2a8_linear_gemv.argtypes = [P, P, I64, I64, F32, P, P, P, I64, P]
        L.w2a8_linear_gemv.restype = I32
        L.w2a4_act_bytes.argtypes = [I64, I64]
        L.w2a4_act_bytes.restype = I64
        L.pack_act_int4.argtypes = [P, I64, I64, P, I64]
        L.pack_act_int4.restype = I32
        L.quant_act_int4.argtypes = [P, I64, I64, P, P, P]
        L.quant_act_int4.restype = I32
        L.w2a4_gemv.argtypes = [P, P, I64, I64, P, P, F32, P, P, I64, P]
        L.w2a4_gemv.restype = I32
        L.w2a4_linear_gemv.argtypes = [P, P, I64, I64, F32, P, P, P, I64, P]
        L.w2a4_linear_gemv.restype = I32
        L.w2a8_gemv_grouped.argtypes = [I32, P, P, I64, P, P, P, P, P, P, I64, P]
        L.w2a8_gemv_grouped.restype = I32
        L.w2a8_linear_gemv_grouped.argtypes = [I32, P, P, I64, P, P, P, P, P, I64, P]
        L.w2a8_linear_gemv_grouped.restype = I32
        for name in ("mx4_act_bytes", "mx4_scale_bytes", "mx4_packed_bytes"):
            getattr(L, name).argtypes = [I64, I64]
            getattr(L, name).restype = I64
        for name, args in (("pack_mx4", [P, P, I64, I64, P, I64]),
                           ("unpack_mx4", [P, I64, I64, I64, P, P]),
                           ("quant_act_mx4", [P, I32, I64, I64, P, P, P]),
                           ("dequant_act_mx4", [P, P, I64, I64, P, I32, P]),
                           ("quant_pack_mx4", [P, I32, I64, I64, P, I64, P]),
                           ("w4mx4_gemm", [P, P, P, I64, I64, I64, P, P, P]),
                           ("w2mx4_gemm", [P, P, P, I64, I64, I64, F32, P, P, P]),
                           ("w4mx4_linear_gemv", [P, P, I32, I64, I64, P, P, P]),
                           ("w2mx4_linear_gemv", [P, P, I32, I64, I64, F32, P, P, P])):
            getattr(L, name).argtypes = args
            getattr(L, name).restype = I32
        L.w4a8_packed_bytes.argtypes = [I64, I64, I64, I32]
        L.w4a8_packed_bytes.restype = I64
        L.w2a8_w4a8_plan.argtypes = [I64, I64, I64, I64, I32, P, P, P, P]
        L.w2a8_w4a8_plan.restype = I32
        L.w2a8_moe_plan.argtypes = [I64, I64, I64, I64, I64, I32, P, P, P]
        L.w2a8_moe_plan.restype = I32
        L.w2a8_tune_moe.argtypes = [I32]
        L.w2a8_tune_moe.restype = I32
        L.w4a8_workspace_bytes.argtypes = [I64, I64, I64]
        L.w4a8_workspace_bytes.restype = I64
        L.w2a8_moe_workspace_bytes.argtypes = [I64] * 5
        L.w2a8_moe_workspace_bytes.restype = I64
        for name, args in (("rmsnorm_quant_int8", [P, P, P, I32, I64, I64, F32, P, P, P, P]),
                           ("pack_w4a8", [P, P, P, I64, I64, I64, P, I64]),
                           ("unpack_w4a8", [P, I64, I64, I64, I64, P, P, P]),
                           ("w4a8_gemm", [P, P, P, I64, I64, I64, I64, I32, I32, P, P, P, I64, P]),
                           ("w2a8_moe", [P, P, P, I32, P, P, P, P, P, P, I64, I64, I64, I64, I64,
                                         I32, I32, P, P, P, I64, P])):
            getattr(L, name).argtypes = args
            getattr(L, name).restype = I32
        L.w2a8_tune_gemv.argtypes = [I32, I32, I32, I32, I32]
        L.w2a8_tune_gemv.restype = I32
        L.w2a8_gemv_plan.argtypes = [I64, I64, I32, P, P, P, P]
        L.w2a8_linear_plan.argtypes = [I64, I64, I32, I32, P, P, P, P, P]
        L.w2a8_linear_plan.restype = I32
        L.w2a8_mx4_plan.argtypes = [I64, I64, I64, I32, I32, I32, P, P, P, P, P]
        L.w2a8_mx4_plan.restype = I32
        L.w2a8_tune_gemv_force.argtypes = [I32, I32, I32, I32, I32]
        L.w2a8_tune_gemv_force.restype = I32
        L.w2a8_tune_gemm.argtypes = [I32]
        L.w2a8_tune_gemm.restype = I32
        L.w2a8_tune_gemm_pipe.argtypes = [I32]
        L.w2a8_tune_gemm_pipe.restype = I32
        L.w2a8_tune_gemm_ring.argtypes = [I32, I32, I32]
        L.w2a8_tune_gemm_ring.restype = I32
        L.w2a8_gemv_plan.restype = I32
        if L.w2a8_layout_version() != LAYOUT_VERSION:
            raise RuntimeError("libw2a8.so layout version does not match the binding")
        _lib = L
        return L


def _check(status: int, where: str):
    if status != 0:
        raise W2A8Error(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _need(t, name, dtype, device=None, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device == "cuda" and not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if device == "cpu" and t.is_cuda:
        raise ValueError(f"{name} must be a host tensor")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


# ---------------------------------------------------------------------------
# sizes
# ---------------------------------------------------------------------------
def layout_version() -> int:
    return int(lib().w2a8_layout_version())


def packed_bytes(N: int, K: int) -> int:
    n = int(lib().w2a8_packed_bytes(N, K))
    if n < 0:
        raise W2A8Error(2, "w2a8_packed_bytes")
    return n


def workspace_bytes(M: int, N: int, K: int) -> int:
    n = int(lib().w2a8_workspace_bytes(M, N, K))
    if n < 0:
        raise W2A8Error(2, "w2a8_workspace_bytes")
    return n


# ---------------------------------------------------------------------------
# offline host steps
# ---------------------------------------------------------------------------
def ternarize_absmean(W: torch.Tensor):
    """W fp32 [N, K] (CPU) -> (wq int8 [N, K] CPU, sw float)."""
    _need(W, "W", torch.float32, "cpu")
    N, K = W.shape
    wq = torch.empty((N, K), dtype=torch.int8)
    sw = torch.zeros(1, dtype=torch.float32)
    _check(lib().w2a8_ternarize_absmean(_ptr(W), N, K, _ptr(wq), _ptr(sw)),
           "w2a8_ternarize_absmean")
    return wq, float(sw[0])


def pack_ternary(w: torch.Tensor) -> torch.Tensor:
    """w int8 [N, K] in {-1,0,1} (CPU) -> packed uint8 [packed_bytes(N, K)] (CPU)."""
    _need(w, "w", torch.int8, "cpu")
    N, K = w.shape
    nb = packed_bytes(N, K)
    out = torch.empty(nb, dtype=torch.uint8)
    _check(lib().pack_ternary(_ptr(w), N, K, _ptr(out), nb), "pack_ternary")
    return out


def unpack_ternary(p: torch.Tensor, N: int, K: int) -> torch.Tensor:
    _need(p, "packed", torch.uint8, "cpu")
    w = torch.empty((N, K), dtype=torch.int8)
    _check(lib().unpack_ternary(_ptr(p), p.numel(), N, K, _ptr(w)), "unpack_ternary")
    return w


# ---------------------------------------------------------------------------
# workspace cache (one zeroed buffer per device and stream)
# ---------------------------------------------------------------------------
class Workspace:
    """Zero-initialised device workspace; each library call leaves it zeroed."""

    _cache = {}
    _lock = threading.Lock()

    @classmethod
    def get(cls, nbytes: int, device: torch.device, stream) -> torch.Tensor | None:
        if nbytes <= 0:
            return None
        key = (device.index, stream.cuda_stream)
        with cls._lock:
            buf = cls._cache.get(key)
            if buf is None or buf.numel() < nbytes:
                with torch.cuda.stream(stream):
                    buf = torch.zeros(max(nbytes, 4096), dtype=torch.uint8, device=device)
                cls._cache[key] = buf
            return buf


def _ws(nbytes, device, stream, workspace):
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8, "cuda")
        return workspace
    s = torch.cuda.current_stream(device) if stream is None else stream
    return Workspace.get(nbytes, device, s)


# ---------------------------------------------------------------------------
# device steps
# ---------------------------------------------------------------------------
def quant_act_int8(x_bf16: torch.Tensor, x_q=None, s_a=None, stream=None):
    """x bf16 [M, K] (device) -> (x_q int8 [M, K], s_a fp32 [M])."""
    _need(x_bf16, "x_bf16", torch.bfloat16, "cuda")
    if x_bf16.dim() == 1:
        x_bf16 = x_bf16.view(1, -1)
    M, K = x_bf16.shape
    if x_q is None:
        x_q = torch.empty((M, K), dtype=torch.int8, device=x_bf16.device)
    if s_a is None:
        s_a = torch.empty(M, dtype=torch.float32, device=x_bf16.device)
    _need(x_q, "x_q", torch.int8, "cuda")
    _need(s_a, "s_a", torch.float32, "cuda")
    if x_q.numel() != M * K or s_a.numel() != M:
        raise ValueError("x_q / s_a have the wrong size")
    _check(lib().quant_act_int8(_ptr(x_bf16), M, K, _ptr(x_q), _ptr(s_a), _stream_handle(stream)),
           "quant_act_int8")
    return x_q, s_a


def w2a8_gemv(w_packed, x, N, K, y_i32=None, s_a=None, s_w=1.0, y_f32=None,
              workspace=None, stream=None):
    """Raw C-ABI call (outputs must be given); returns nothing."""
    _need(w_packed, "w_packed", torch.uint8, "cuda")
    _need(x, "x", torch.int8, "cuda")
    if x.numel() != K:
        raise ValueError("x must have K elements")
    if w_packed.numel() < packed_bytes(N, K):
        raise ValueError("w_packed is smaller than packed_bytes(N, K)")
    for t, nm, dt in ((y_i32, "y_i32", torch.int32), (y_f32, "y_f32", torch.float32)):
        if t is not None:
            _need(t, nm, dt, "cuda")
            if t.numel() != N:
                raise ValueError(f"{nm} must have N elements")
    if s_a is not None:
        _need(s_a, "s_a", torch.float32, "cuda")
    need = workspace_bytes(1, N, K)
    ws = _ws(need, x.device, stream, workspace)
    _check(lib().w2a8_gemv(_ptr(w_packed), _ptr(x), N, K, _ptr(y_i32), _ptr(s_a),
                           ctypes.c_float(s_w), _ptr(y_f32), _ptr(ws),
                           0 if ws is None else ws.numel(), _stream_handle(stream)),
           "w2a8_gemv")


def w2a8_gemv_noalloc(w_packed, x, N, K, y_i32=None, s_a=None, s_w=1.0, y_f32=None,
                      stream=None):
    """Raw C-ABI call: the GEMV with the library's static scratch instead of a
    workspace (allocates nothing); returns nothing."""
    _need(w_packed, "w_packed", torch.uint8, "cuda")
    _need(x, "x", torch.int8, "cuda")
    if x.numel() != K:
        raise ValueError("x must have K elements")
    if w_packed.numel() < packed_bytes(N, K):
        raise ValueError("w_packed is smaller than packed_bytes(N, K)")
    for t, nm, dt in ((y_i32, "y_i32", torch.int32), (y_f32, "y_f32", torch.float32)):
        if t is not None:
            _need(t, nm, dt, "cuda")
            if t.numel() != N:
                raise ValueError(f"{nm} must have N elements")
    if s_a is not None:
        _need(s_a, "s_a", torch.float32, "cuda")
    _check(lib().w2a8_gemv_noalloc(_ptr(w_packed), _ptr(x), N, K, _ptr(y_i32), _ptr(s_a),
                                   ctypes.c_float(s_w), _ptr(y_f32), _stream_handle(stream)),
           "w2a8_gemv_noalloc")


def w2a8_gemm(w_packed, x, M, N, K, y_i32=None, s_a=None, s_w=1.0, y_f32=None,
              workspace=None, stream=None):
    """Raw C-ABI call (outputs must be given); returns nothing."""
    _need(w_packed, "w_packed", torch.uint8, "cuda")
    _need(x, "x", torch.int8, "cuda")
    if x.numel() != M * K:
        raise ValueError("x must have M*K elements")
    if w_packed.numel() < packed_bytes(N, K):
        raise ValueError("w_packed is smaller than packed_bytes(N, K)")
    for t, nm, dt in ((y_i32, "y_i32", torch.int32), (y_f32, "y_f32", torch.float32)):
        if t is not None:
            _need(t, nm, dt, "cuda")
            if t.numel() != M * N:
                raise ValueError(f"{nm} must have M*N elements")
    if s_a is not None:
        _need(s_a, "s_a", torch.float32, "cuda")
        if s_a.numel() != M:
            raise ValueError("s_a must have M elements")
    need = workspace_bytes(M, N, K)
    ws = _ws(need, x.device, stream, workspace)
    _check(lib().w2a8_gemm(_ptr(w_packed), _ptr(x), M, N, K, _ptr(y_i32), _ptr(s_a),
                           ctypes.c_float(s_w), _ptr(y_f32), _ptr(ws),
                           0 if ws is None else ws.numel(), _stream_handle(stream)),
           "w2a8_gemm")


def w2a8_linear_gemv(w_packed, x_bf16, N, K, s_w, y_f32, y_i32=None, workspace=None,
                     stream=None):
    """Raw C-ABI call: fused quantize + GEMV + fp32 epilogue for one token."""
    _need(w_packed, "w_packed", torch.uint8, "cuda")
    if x_bf16.dtype not in (torch.bfloat16, torch.int16, torch.uint16) or not x_bf16.is_cuda:
        raise TypeError("x_bf16 must be a bfloat16 (or 16-bit bit pattern) CUDA tensor")
    if not x_bf16.is_contiguous() or x_bf16.numel() != K:
        raise ValueError("x_bf16 must be contiguous with K elements")
    if w_packed.numel() < packed_bytes(N, K):
        raise ValueError("w_packed is smaller than packed_bytes(N, K)")
    _need(y_f32, "y_f32", torch.float32, "cuda")
    if y_f32.numel() != N:
        raise ValueError("y_f32 must have N elements")
    if y_i32 is not None:
        _need(y_i32, "y_i32", torch.int32, "cuda")
        if y_i32.numel() != N:
            raise ValueError("y_i32 must have N elements")
    ws = _ws(workspace_bytes(1, N, K), x_bf16.device, stream, workspace)
    _check(lib().w2a8_linear_gemv(_ptr(w_packed), _ptr(x_bf16), N, K, ctypes.c_float(s_w),
                                  _ptr(y_f32), _ptr(y_i32), _ptr(ws),
                                  0 if ws is None else ws.numel(), _stream_handle(stream)),
           "w2a8_linear_gemv")


# ---------------------------------------------------------------------------
# W2A4 variant: int4 activations in the A4I layout (see include/w2a8.h)
# ---------------------------------------------------------------------------
def act4_bytes(M: int, K: int) -> int:
    v = int(lib().w2a4_act_bytes(M, K))
    if v < 0:
        raise ValueError("M or K out of range")
    return v


def pack_act_int4(q: torch.Tensor) -> torch.Tensor:
    """Host int8 [M, K] (values -8..7) -> host uint8 [act4_bytes(M, K)] (A4I layout)."""
    q2 = q.view(1, -1) if q.dim() == 1 else q
    _need(q2, "q", torch.int8, "cpu")
    M, K = q2.shape
    out = torch.empty(act4_bytes(M, K), dtype=torch.uint8)
    _check(lib().pack_act_int4(_ptr(q2), M, K, _ptr(out), out.numel()), "pack_act_int4")
    return out


def quant_act_int4(x_bf16: torch.Tensor, x_q4=None, s_a=None, stream=None):
    """x bf16 [M, K] (device) -> (A4I bytes uint8 [act4_bytes(M, K)], s_a fp32 [M])."""
    _need(x_bf16, "x_bf16", torch.bfloat16, "cuda")
    x2 = x_bf16.view(1, -1) if x_bf16.dim() == 1 else x_bf16
    M, K = x2.shape
    if x_q4 is None:
        x_q4 = torch.empty(act4_bytes(M, K), dtype=torch.uint8, device=x2.device)
    if s_a is None:
        s_a = torch.empty(M, dtype=torch.float32, device=x2.device)
    _need(x_q4, "x_q4", torch.uint8, "cuda")
    _need(s_a, "s_a", torch.float32, "cuda")
    if x_q4.numel() < act4_bytes(M, K) or s_a.numel() != M:
        raise ValueError("x_q4 / s_a have the wrong size")
    _check(lib().quant_act_int4(_ptr(x2), M, K, _ptr(x_q4), _ptr(s_a), _stream_handle(stream)),
           "quant_act_int4")
    return x_q4, s_a


def w2a4_gemv(w_packed, x_q4, N, K, y_i32=None, s_a=None, s_w=1.0, y_f32=None,
              workspace=None, stream=None):
    """Raw C-ABI call: W2A4 GEMV over one A4I activation row; returns nothing."""
    _need(w_packed, "w_packed", torch.uint8, "cuda")
    _need(x_q4, "x_q4", torch.uint8, "cuda")
    if x_q4.numel() < act4_bytes(1, K):
        raise ValueError("x_q4 must hold act4_bytes(1, K) bytes")
    if w_packed.numel() < packed_bytes(N, K):
        raise ValueError("w_packed is smaller than packed_bytes(N, K)")
    for t, nm, dt in ((y_i32, "y_i32", torch.int32), (y_f32, "y_f32", torch.float32)):
        if t is not None:
            _need(t, nm, dt, "cuda")
            if t.numel() != N:
                raise ValueError(f"{nm} must have N elements")
    if s_a is not None:
        _need(s_a, "s_a", torch.float32, "cuda")
    ws = _ws(workspace_bytes(1, N, K), x_q4.device, stream, workspace)
    _check(lib().w2a4_gemv(_ptr(w_packed), _ptr(x_q4), N, K, _ptr(y_i32), _ptr(s_a),
                           ctypes.c_float(s_w), _ptr(y_f32), _ptr(ws),
                           0 if ws is None else ws.numel(), _stream_handle(stream)),
           "w2a4_gemv")


def w2a4_linear_gemv(w_packed, x_bf16, N, K, s_w, y_f32, y_i32=None, workspace=None,
                     stream=None):
    """Raw C-ABI call: fused int4 quantize + W2A4 GEMV + fp32 epilogue for one token."""
    _need(w_packed, "w_packed", torch.uint8, "cuda")
    if x_bf16.dtype not in (torch.bfloat16, torch.int16, torch.uint16) or not x_bf16.is_cuda:
        raise TypeError("x_bf16 must be a bfloat16 (or 16-bit bit pattern) CUDA tensor")
    if not x_bf16.is_contiguous() or x_bf16.numel() != K:
        raise ValueError("x_bf16 must be contiguous with K elements")
    if w_packed.numel() < packed_bytes(N, K):
        raise ValueError("w_packed is smaller than packed_bytes(N, K)")
    _need(y_f32, "y_f32", torch.float32, "cuda")
    if y_f32.numel() != N:
        raise ValueError("y_f32 must have N elements")
    if y_i32 is not None:
        _need(y_i32, "y_i32", torch.int32, "cuda")
        if y_i32.numel() != N:
            raise ValueError("y_i32 must have N elements")
    ws = _ws(workspace_bytes(1, N, K), x_bf16.device, stream, workspace)
    _check(lib().w2a4_linear_gemv(_ptr(w_packed), _ptr(x_bf16), N, K, ctypes.c_float(s_w),
                                  _ptr(y_f32), _ptr(y_i32), _ptr(ws),
                                  0 if ws is None else ws.numel(), _stream_handle(stream)),
           "w2a4_linear_gemv")


def linear_a4(x_bf16, w_packed, s_w, N, K, stream=None, fused=True):
    """W2A4 linear layer for one token -> fp32 [1, N].  fused=True:
    w2a4_linear_gemv (one launch); otherwise quant_act_int4, then w2a4_gemv
    with the fp32 epilogue (two launches, no host synchronisation).  Both
    routes give bit-identical results."""
    if fused:
        y = torch.empty((1, N), dtype=torch.float32, device=x_bf16.device)
        w2a4_linear_gemv(w_packed, x_bf16.reshape(-1), N, K, s_w, y.view(-1), stream=stream)
        return y
    xq4, sa = quant_act_int4(x_bf16.reshape(1, -1), stream=stream)
    y = torch.empty((1, N), dtype=torch.float32, device=x_bf16.device)
    w2a4_gemv(w_packed, xq4, N, K, s_a=sa, s_w=s_w, y_f32=y.view(-1), stream=stream)
    return y


MAX_GROUPS = 8


def _host_array(ctype, values):
    return (ctype * len(values))(*values)


def _grouped_args(w_packed, Ns, K, s_w, y_i32, y_f32):
    G = len(w_packed)
    if not (1 <= G <= MAX_GROUPS) or len(Ns) != G or len(s_w) != G:
        raise ValueError(f"need 1..{MAX_GROUPS} projections with one N and one s_w each")
    for g, (w, n) in enumerate(zip(w_packed, Ns)):
        _need(w, f"w_packed[{g}]", torch.uint8, "cuda")
        if w.numel() < packed_bytes(n, K):
            raise ValueError(f"w_packed[{g}] is smaller than packed_bytes(N[{g}], K)")
    arrays = []
    for ys, nm, dt in ((y_i32, "y_i32", torch.int32), (y_f32, "y_f32", torch.float32)):
        if ys is None:
            arrays.append(None)
            continue
        if len(ys) != G:
            raise ValueError(f"{nm} must have one entry per projection")
        for g, (y, n) in enumerate(zip(ys, Ns)):
            if y is not None:
                _need(y, f"{nm}[{g}]", dt, "cuda")
                if y.numel() != n:
                    raise ValueError(f"{nm}[{g}] must have N[{g}] elements")
        arrays.append(_host_array(ctypes.c_void_p, [None if y is None else y.data_ptr() for y in ys]))
    need = sum(workspace_bytes(1, n, K) for n in Ns)
    return (G, _host_array(ctypes.c_void_p, [w.data_ptr() for w in w_packed]),
            _host_array(ctypes.c_int64, list(Ns)), _host_array(ctypes.c_float, list(s_w)),
            arrays[0], arrays[1], need)


def w2a8_gemv_grouped(w_packed, x, Ns, K, s_w, y_i32=None, y_f32=None, s_a=None,
                      workspace=None, stream=None):
    """Raw C-ABI call: several projections (lists of equal length) sharing one
    int8 activation row x [K], in one launch; returns nothing."""
    _need(x, "x", torch.int8, "cuda")
    if x.numel() != K:
        raise ValueError("x must have K elements")
    if s_a is not None:
        _need(s_a, "s_a", torch.float32, "cuda")
    G, wp, n_arr, sw_arr, yi_arr, yf_arr, need = _grouped_args(w_packed, Ns, K, s_w, y_i32, y_f32)
    ws = _ws(need, x.device, stream, workspace)
    _check(lib().w2a8_gemv_grouped(G, wp, n_arr, K, _ptr(x), _ptr(s_a), sw_arr, yi_arr, yf_arr,
                                   _ptr(ws), 0 if ws is None else ws.numel(),
                                   _stream_handle(stream)),
           "w2a8_gemv_grouped")


def w2a8_linear_gemv_grouped(w_packed, x_bf16, Ns, K, s_w, y_f32, y_i32=None, workspace=None,
                             stream=None):
    """Raw C-ABI call: quantize one bf16 token and apply several projections
    to it, in one launch; returns nothing."""
    if x_bf16.dtype not in (torch.bfloat16, torch.int16, torch.uint16) or not x_bf16.is_cuda:
        raise TypeError("x_bf16 must be a bfloat16 (or 16-bit bit pattern) CUDA tensor")
    if not x_bf16.is_contiguous() or x_bf16.numel() != K:
        raise ValueError("x_bf16 must be contiguous with K elements")
    G, wp, n_arr, sw_arr, yi_arr, yf_arr, need = _grouped_args(w_packed, Ns, K, s_w, y_i32, y_f32)
    ws = _ws(need, x_bf16.device, stream, workspace)
    _check(lib().w2a8_linear_gemv_grouped(G, wp, n_arr, K, _ptr(x_bf16), sw_arr, yf_arr, yi_arr,
                                          _ptr(ws), 0 if ws is None else ws.numel(),
                                          _stream_handle(stream)),
           "w2a8_linear_gemv_grouped")


def linear_grouped(x_bf16, w_packed, s_w, Ns, K, stream=None):
    """Several W2A8 linear layers applied to one bf16 token (one launch):
    returns a list of fp32 [1, N_g] outputs."""
    ys = [torch.empty((1, n), dtype=torch.float32, device=x_bf16.device) for n in Ns]
    w2a8_linear_gemv_grouped(w_packed, x_bf16.reshape(-1), Ns, K, s_w, [y.view(-1) for y in ys],
                             stream=stream)
    return ys


def gemv(w_packed, x, N, K, *, out_i32=True, s_a=None, s_w=1.0, stream=None):
    """y_i32 [N] (and y_f32 [N] when s_a is given) for one int8 activation row."""
    y_i32 = torch.empty(N, dtype=torch.int32, device=x.device) if out_i32 else None
    y_f32 = torch.empty(N, dtype=torch.float32, device=x.device) if s_a is not None else None
    w2a8_gemv(w_packed, x, N, K, y_i32=y_i32, s_a=s_a, s_w=s_w, y_f32=y_f32, stream=stream)
    return y_i32 if y_f32 is None else (y_i32, y_f32)


def gemm(w_packed, x, N, K, *, out_i32=True, s_a=None, s_w=1.0, stream=None):
    """Y_i32 [M, N] (and Y_f32 when s_a is given) for int8 activations [M, K]."""
    M = x.shape[0]
    y_i32 = torch.empty((M, N), dtype=torch.int32, device=x.device) if out_i32 else None
    y_f32 = torch.empty((M, N), dtype=torch.float32, device=x.device) if s_a is not None else None
    w2a8_gemm(w_packed, x, M, N, K, y_i32=y_i32, s_a=s_a, s_w=s_w, y_f32=y_f32, stream=stream)
    return y_i32 if y_f32 is None else (y_i32, y_f32)


def linear(x_bf16, w_packed, s_w, N, K, stream=None, fused=True):
    """Full W2A8 linear layer: bf16 activations [M, K] -> fp32 [M, N].

    M == 1 with fused=True: w2a8_linear_gemv (one launch).  Otherwise
    quant_act_int8, then w2a8_gemv (M == 1) or w2a8_gemm (M > 1) with the
    fp32 epilogue, all enqueued on one stream with no host synchronisation.
    Both routes give bit-identical results.
    """
    x2 = x_bf16.view(1, -1) if x_bf16.dim() == 1 else x_bf16
    M = x2.shape[0]
    if M == 1 and fused:
        y = torch.empty((1, N), dtype=torch.float32, device=x2.device)
        w2a8_linear_gemv(w_packed, x2.reshape(-1), N, K, s_w, y.view(-1), stream=stream)
        return y
    xq, sa = quant_act_int8(x2, stream=stream)
    y = torch.empty((M, N), dtype=torch.float32, device=x2.device)
    if M == 1:
        w2a8_gemv(w_packed, xq.view(-1), N, K, s_a=sa, s_w=s_w, y_f32=y.view(-1), stream=stream)
    else:
        w2a8_gemm(w_packed, xq, M, N, K, s_a=sa, s_w=s_w, y_f32=y, stream=stream)
    return y


# ---------------------------------------------------------------------------
# MX4: 4-bit floats in blocks of 32 with a power-of-two scale (see
# include/w2a8_mx4.h)
# ---------------------------------------------------------------------------
_MX4_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


@functools.lru_cache(maxsize=4096)
def _mx4_size(name, a, b):
    v = int(getattr(lib(), name)(a, b))
    if v < 0:
        raise W2A8Error(2, name)
    return v


def mx4_act_bytes(M: int, K: int) -> int:
    """Code bytes of M rows of K values (MX4R)."""
    return _mx4_size("mx4_act_bytes", M, K)


def mx4_scale_bytes(M: int, K: int) -> int:
    """Scale bytes of M rows of K values (MX4R)."""
    return _mx4_size("mx4_scale_bytes", M, K)


def mx4_packed_bytes(N: int, K: int) -> int:
    """Bytes of packed MX4 weights (MX16x128)."""
    return _mx4_size("mx4_packed_bytes", N, K)


def pack_mx4(codes: torch.Tensor, scales: torch.Tensor, N: int, K: int) -> torch.Tensor:
    """Interchange form (CPU): codes uint8 [N, ceil(K/2)], two values a byte, the lower k in
    the lower half, and scales uint8 [N, ceil(K/32)] -> packed uint8 [mx4_packed_bytes] (CPU)."""
    _need(codes, "codes", torch.uint8, "cpu", (N, -(-K // 2)))
    _need(scales, "scales", torch.uint8, "cpu", (N, -(-K // 32)))
    out = torch.empty(mx4_packed_bytes(N, K), dtype=torch.uint8)
    _check(lib().pack_mx4(_ptr(codes), _ptr(scales), N, K, _ptr(out), out.numel()), "pack_mx4")
    return out


def unpack_mx4(packed: torch.Tensor, N: int, K: int):
    """Packed MX4 weights (CPU) -> (codes, scales) in the interchange form."""
    _need(packed, "packed", torch.uint8, "cpu")
    mx4_packed_bytes(N, K)
    codes = torch.empty((N, -(-K // 2)), dtype=torch.uint8)
    scales = torch.empty((N, -(-K // 32)), dtype=torch.uint8)
    _check(lib().unpack_mx4(_ptr(packed), packed.numel(), N, K, _ptr(codes), _ptr(scales)),
           "unpack_mx4")
    return codes, scales


# At one row the calls below cost the host more than their kernels take, so
# each argument is checked once and by one expression, sizes are remembered,
# and outputs made here are not checked again (8.1 us a product call before,
# 3.8 of them ctypes, launch and kernel).
@functools.lru_cache(maxsize=4096)
def _mx4_sizes(M, N, K, ternary):
    """Bytes of the rows' codes and scales and of the weights of a product."""
    return (mx4_act_bytes(M, K), mx4_scale_bytes(M, K),
            _mx4_size("w2a8_packed_bytes" if ternary else "mx4_packed_bytes", N, K))


def _mx4_gpu(t, name):
    """The index of a tensor's device, which has to be the current GPU."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be a device tensor")
    if index != torch._C._cuda_getDevice():               # torch.cuda.current_device()
        raise ValueError(f"{name} is on {t.device}, which is not the current device")
    return index


def _mx4_ptr(t, name, index, dtype, least, most=None):
    """The address of a contiguous tensor of `dtype` on device `index` with `least` elements
    or more (`most` at most)."""
    if isinstance(t, torch.Tensor):
        if (t.dtype is dtype and t.get_device() == index and t.is_contiguous()
                and least <= t.numel() and (most is None or t.numel() <= most)):
            return t.data_ptr()
    else:
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the first argument on cuda:{index}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must have {'at least ' if most is None else ''}{least} elements, "
                     f"got {t.numel()}")


def _mx4_type(t, name):
    """The w2a8_mx4_type of a contiguous float tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    code = _MX4_TYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return code


def _mx4_stream(stream, index):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)   # current_stream(index).cuda_stream
    if stream.device.index != index:
        raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{index}")
    return stream.cuda_stream


def _mx4_empty(like, shape, dtype, stream):
    """Uninitialised memory that belongs to the stream of the call."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _mx4_rows(x, name):
    if x.dim() == 1:
        return 1, x.shape[0]
    if x.dim() != 2:
        raise ValueError(f"{name} must be [M, K] or [K]")
    return x.shape


def quant_act_mx4(x: torch.Tensor, x_q=None, x_s=None, stream=None):
    """x fp32, bf16 or fp16 [M, K] (or [K]: one row; device) -> (x_q uint8 [M, 64 * KT] codes,
    x_s uint8 [M, 16 * KU] scale bytes), the MX4R layout.  x_q and x_s may be given (any shape
    of at least mx4_act_bytes / mx4_scale_bytes elements)."""
    code, dev = _mx4_type(x, "x"), _mx4_gpu(x, "x")
    M, K = _mx4_rows(x, "x")
    nq, ns = mx4_act_bytes(M, K), mx4_scale_bytes(M, K)
    if x_q is None:
        x_q = _mx4_empty(x, (M, nq // M), torch.uint8, stream)
        pq = x_q.data_ptr()
    else:
        pq = _mx4_ptr(x_q, "x_q", dev, torch.uint8, nq)
    if x_s is None:
        x_s = _mx4_empty(x, (M, ns // M), torch.uint8, stream)
        ps = x_s.data_ptr()
    else:
        ps = _mx4_ptr(x_s, "x_s", dev, torch.uint8, ns)
    st = lib().quant_act_mx4(x.data_ptr(), code, M, K, pq, ps, _mx4_stream(stream, dev))
    if st:
        raise W2A8Error(st, "quant_act_mx4")
    return x_q, x_s


def _mx4_count(x_q):
    """The rows of a 2-d x_q."""
    if not isinstance(x_q, torch.Tensor):
        raise TypeError("x_q must be a torch.Tensor")
    if x_q.dim() != 2:
        raise ValueError("x_q must be [M, bytes of a row] where M is not given")
    return x_q.shape[0]


def _mx4_scale_rows(x_s, row):
    """Refuses rows of x_s that are not `row` bytes (a flat x_s is a buffer)."""
    if x_s.dim() > 1 and x_s.shape[-1] != row:
        raise ValueError(f"x_s must have rows of {row} bytes, got {x_s.shape[-1]}")


def dequant_act_mx4(x_q, x_s, K: int, M=None, dtype=torch.float32, y=None, stream=None):
    """MX4R rows -> their values [M, K] in fp32, bf16 or fp16 (device).  M defaults to the
    rows of x_q [M, mx4_act_bytes(1, K)] (x_s: [M, mx4_scale_bytes(1, K)], or flat); with M
    given, x_q and x_s are buffers of at least M rows.  y may be given (M * K elements of
    dtype)."""
    counted = M is None
    if counted:
        M = _mx4_count(x_q)
    dev = _mx4_gpu(x_q, "x_q")
    code = _MX4_TYPES.get(dtype)
    if code is None:
        raise TypeError(f"dtype must be float32, bfloat16 or float16, got {dtype}")
    na, ns = mx4_act_bytes(M, K), mx4_scale_bytes(M, K)
    pq = _mx4_ptr(x_q, "x_q", dev, torch.uint8, na, na if counted else None)
    ps = _mx4_ptr(x_s, "x_s", dev, torch.uint8, ns)
    if counted and x_s.numel() != ns:
        _mx4_scale_rows(x_s, ns // M)
    if y is None:
        y = _mx4_empty(x_q, (M, K), dtype, stream)
        py = y.data_ptr()
    else:
        py = _mx4_ptr(y, "y", dev, dtype, M * K, M * K)
    st = lib().dequant_act_mx4(pq, ps, M, K, py, code, _mx4_stream(stream, dev))
    if st:
        raise W2A8Error(st, "dequant_act_mx4")
    return y


def quant_pack_mx4(W: torch.Tensor, packed=None, stream=None) -> torch.Tensor:
    """Float weights [N, K] (device) -> packed MX4 weights uint8 [mx4_packed_bytes(N, K)]."""
    code, dev = _mx4_type(W, "W"), _mx4_gpu(W, "W")
    if W.dim() != 2:
        raise ValueError("W must be [N, K]")
    N, K = W.shape
    nb = mx4_packed_bytes(N, K)
    if packed is None:
        packed = _mx4_empty(W, (nb,), torch.uint8, stream)
    _check(lib().quant_pack_mx4(W.data_ptr(), code, N, K,
                                _mx4_ptr(packed, "packed", dev, torch.uint8, nb), packed.numel(),
                                _mx4_stream(stream, dev)), "quant_pack_mx4")
    return packed


def _mx4_outputs(y_f32, y_bf16, dev, count):
    return (None if y_f32 is None else _mx4_ptr(y_f32, "y_f32", dev, torch.float32, count, count),
            None if y_bf16 is None else _mx4_ptr(y_bf16, "y_bf16", dev, torch.bfloat16, count, count))


def _mx4_new(like, dtype, shape, stream):
    """A new output and its two addresses (y_f32, y_bf16), one of them None."""
    if dtype is not torch.float32 and dtype is not torch.bfloat16:
        raise TypeError(f"out_dtype must be float32 or bfloat16, got {dtype}")
    y = _mx4_empty(like, shape, dtype, stream)
    return (y, y.data_ptr(), None) if dtype is torch.float32 else (y, None, y.data_ptr())


def _mx4_gemm(w_packed, x_q, x_s, M, N, K, s_w, yf, yb, dev, stream, counted):
    """A product (s_w None: MX4 weights) into the addresses yf and yb."""
    na, ns, nw = _mx4_sizes(M, N, K, s_w is not None)
    pw = _mx4_ptr(w_packed, "w_packed", dev, torch.uint8, nw)
    # Rows that were counted have to be rows of K values: those of a longer K are a larger
    # buffer, but lie elsewhere in it.
    pq = _mx4_ptr(x_q, "x_q", dev, torch.uint8, na, na if counted else None)
    ps = _mx4_ptr(x_s, "x_s", dev, torch.uint8, ns)
    if counted and x_s.numel() != ns:
        _mx4_scale_rows(x_s, ns // M)
    if s_w is None:
        st = lib().w4mx4_gemm(pw, pq, ps, M, N, K, yf, yb, _mx4_stream(stream, dev))
    else:
        st = lib().w2mx4_gemm(pw, pq, ps, M, N, K, s_w, yf, yb, _mx4_stream(stream, dev))
    if st:
        raise W2A8Error(st, "w4mx4_gemm" if s_w is None else "w2mx4_gemm")


def _mx4_gemv(w_packed, x, code, N, K, s_w, yf, yb, dev, stream):
    """A one-launch layer (s_w None: MX4 weights) into the addresses yf and yb."""
    pw = _mx4_ptr(w_packed, "w_packed", dev, torch.uint8, _mx4_sizes(1, N, K, s_w is not None)[2])
    if s_w is None:
        st = lib().w4mx4_linear_gemv(pw, x.data_ptr(), code, N, K, yf, yb, _mx4_stream(stream, dev))
    else:
        st = lib().w2mx4_linear_gemv(pw, x.data_ptr(), code, N, K, s_w, yf, yb,
                                     _mx4_stream(stream, dev))
    if st:
        raise W2A8Error(st, "w4mx4_linear_gemv" if s_w is None else "w2mx4_linear_gemv")


def w4mx4_gemm(w_packed, x_q, x_s, M, N, K, y_f32=None, y_bf16=None, stream=None):
    """Raw C-ABI call: MX4 rows times MX4 weights (outputs must be given); returns nothing."""
    dev = _mx4_gpu(x_q, "x_q")
    yf, yb = _mx4_outputs(y_f32, y_bf16, dev, M * N)
    _mx4_gemm(w_packed, x_q, x_s, M, N, K, None, yf, yb, dev, stream, False)


def w2mx4_gemm(w_packed, x_q, x_s, M, N, K, s_w=1.0, y_f32=None, y_bf16=None, stream=None):
    """Raw C-ABI call: MX4 rows times packed ternary weights; returns nothing."""
    dev = _mx4_gpu(x_q, "x_q")
    yf, yb = _mx4_outputs(y_f32, y_bf16, dev, M * N)
    _mx4_gemm(w_packed, x_q, x_s, M, N, K, float(s_w), yf, yb, dev, stream, False)


def w4mx4_linear_gemv(w_packed, x, N, K, y_f32=None, y_bf16=None, stream=None):
    """Raw C-ABI call: one float row, rounded to MX4 and multiplied in one launch."""
    code, dev = _mx4_type(x, "x"), _mx4_gpu(x, "x")
    if x.numel() != K:
        raise ValueError("x must have K elements")
    yf, yb = _mx4_outputs(y_f32, y_bf16, dev, N)
    _mx4_gemv(w_packed, x, code, N, K, None, yf, yb, dev, stream)


def w2mx4_linear_gemv(w_packed, x, N, K, s_w=1.0, y_f32=None, y_bf16=None, stream=None):
    """Raw C-ABI call: w4mx4_linear_gemv with packed ternary weights."""
    code, dev = _mx4_type(x, "x"), _mx4_gpu(x, "x")
    if x.numel() != K:
        raise ValueError("x must have K elements")
    yf, yb = _mx4_outputs(y_f32, y_bf16, dev, N)
    _mx4_gemv(w_packed, x, code, N, K, float(s_w), yf, yb, dev, stream)


def gemm_w4mx4(w_packed, x_q, x_s, N, K, out_dtype=torch.float32, stream=None):
    """MX4R rows, x_q [M, mx4_act_bytes(1, K)] and x_s [M, mx4_scale_bytes(1, K)] (or flat),
    times MX4 weights -> fp32 or bf16 [M, N]."""
    M, dev = _mx4_count(x_q), _mx4_gpu(x_q, "x_q")
    y, yf, yb = _mx4_new(x_q, out_dtype, (M, N), stream)
    _mx4_gemm(w_packed, x_q, x_s, M, N, K, None, yf, yb, dev, stream, True)
    return y


def gemm_w2mx4(w_packed, x_q, x_s, s_w, N, K, out_dtype=torch.float32, stream=None):
    """MX4R rows, x_q [M, mx4_act_bytes(1, K)] and x_s [M, mx4_scale_bytes(1, K)] (or flat),
    times ternary weights -> fp32 or bf16 [M, N]."""
    M, dev = _mx4_count(x_q), _mx4_gpu(x_q, "x_q")
    y, yf, yb = _mx4_new(x_q, out_dtype, (M, N), stream)
    _mx4_gemm(w_packed, x_q, x_s, M, N, K, float(s_w), yf, yb, dev, stream, True)
    return y


def _mx4_linear(x, w_packed, s_w, N, K, out_dtype, stream, fused):
    code, dev = _mx4_type(x, "x"), _mx4_gpu(x, "x")
    M, k = _mx4_rows(x, "x")
    if k != K:
        raise ValueError(f"x must have rows of {K} values, got {k}")
    y, yf, yb = _mx4_new(x, out_dtype, (M, N), stream)
    if M == 1 and fused:
        _mx4_gemv(w_packed, x, code, N, K, s_w, yf, yb, dev, stream)
    else:
        x_q, x_s = quant_act_mx4(x, stream=stream)
        _mx4_gemm(w_packed, x_q, x_s, M, N, K, s_w, yf, yb, dev, stream, False)
    return y


def linear_w4mx4(x, w_packed, N, K, out_dtype=torch.float32, stream=None, fused=True):
    """Linear layer with MX4 weights: float rows [M, K] (or [K]) -> fp32 or bf16 [M, N].

    M == 1 with fused=True: w4mx4_linear_gemv (one launch).  Otherwise quant_act_mx4, then
    w4mx4_gemm.  Both routes give bit-identical results."""
    return _mx4_linear(x, w_packed, None, N, K, out_dtype, stream, fused)


def linear_w2mx4(x, w_packed, s_w, N, K, out_dtype=torch.float32, stream=None, fused=True):
    """Linear layer with packed ternary weights and MX4 activations (as linear_w4mx4)."""
    return _mx4_linear(x, w_packed, float(s_w), N, K, out_dtype, stream, fused)


# ---------------------------------------------------------------------------
# Around the ternary layers: norm into int8 rows, 4-bit weights with group
# scales, mixture of ternary experts (see include/w2a8_block.h)
# ---------------------------------------------------------------------------
def rmsnorm_quant_int8(x: torch.Tensor, weight=None, residual=None, eps: float = 1e-5, x_q=None,
                       s_a=None, h=None, stream=None):
    """Root-mean-square norm of x (+ residual), fp32, bf16 or fp16 [M, K] (or [K]: one row;
    device), times weight [K], into int8 rows: (x_q int8 [M, K], s_a fp32 [M], h).

    h is x + residual in their type, which the next block adds to (x itself without a
    residual); h=residual or h=x writes it in place.  x_q * s_a is the normalised row."""
    code, dev = _mx4_type(x, "x"), _mx4_gpu(x, "x")
    M, K = _mx4_rows(x, "x")
    dtype, n = x.dtype, M * K
    pw = None if weight is None else _mx4_ptr(weight, "weight", dev, dtype, K, K)
    if residual is None:
        if h is not None:
            raise ValueError("h is given without a residual")
        h, pr, ph = x, None, None
    else:
        pr = _mx4_ptr(residual, "residual", dev, dtype, n, n)
        if h is None:
            h = torch.empty_like(x) if stream is None else _mx4_empty(x, x.shape, dtype, stream)
            ph = h.data_ptr()
        else:
            ph = _mx4_ptr(h, "h", dev, dtype, n, n)
    if x_q is None:
        x_q = _mx4_empty(x, (M, K), torch.int8, stream)
        pq = x_q.data_ptr()
    else:
        pq = _mx4_ptr(x_q, "x_q", dev, torch.int8, n, n)
    if s_a is None:
        s_a = _mx4_empty(x, (M,), torch.float32, stream)
        ps = s_a.data_ptr()
    else:
        ps = _mx4_ptr(s_a, "s_a", dev, torch.float32, M, M)
    st = lib().rmsnorm_quant_int8(x.data_ptr(), pr, pw, code, M, K, eps, ph, pq, ps,
                                  _mx4_stream(stream, dev))
    if st:
        raise W2A8Error(st, "rmsnorm_quant_int8")
    return x_q, s_a, h


@functools.lru_cache(maxsize=4096)
def w4a8_packed_bytes(N: int, K: int, group: int, zeros: bool = False) -> int:
    """Bytes of packed 4-bit weights with group scales (W4T16x128)."""
    v = int(lib().w4a8_packed_bytes(N, K, group, int(bool(zeros))))
    if v < 0:
        raise W2A8Error(2, "w4a8_packed_bytes")
    return v


def _w4_scale_type(dtype):
    if dtype is not torch.float16 and dtype is not torch.bfloat16:
        raise TypeError(f"scales must be float16 or bfloat16, got {dtype}")
    return _MX4_TYPES[dtype]


def pack_w4a8(codes: torch.Tensor, scales: torch.Tensor, N: int, K: int, group: int,
              zeros=None) -> torch.Tensor:
    """Interchange form (CPU): codes uint8 [N, ceil(K/2)], two values a byte, the lower k in
    the lower half, scales fp16 or bf16 [N, ceil(K/group)] and zeros uint8 of that shape, or
    None (the zero point is 8) -> packed uint8 [w4a8_packed_bytes] (CPU)."""
    out = torch.empty(w4a8_packed_bytes(N, K, group, zeros is not None), dtype=torch.uint8)
    groups = -(-K // group)
    _need(codes, "codes", torch.uint8, "cpu", (N, -(-K // 2)))
    if not isinstance(scales, torch.Tensor):
        raise TypeError("scales must be a torch.Tensor")
    _w4_scale_type(scales.dtype)
    _need(scales, "scales", scales.dtype, "cpu", (N, groups))
    if zeros is not None:
        _need(zeros, "zeros", torch.uint8, "cpu", (N, groups))
    _check(lib().pack_w4a8(_ptr(codes), _ptr(scales), _ptr(zeros), N, K, group, _ptr(out),
                           out.numel()), "pack_w4a8")
    return out


def unpack_w4a8(packed: torch.Tensor, N: int, K: int, group: int, scale_dtype=torch.float16,
                zeros: bool = False):
    """Packed 4-bit weights (CPU) -> (codes, scales, zeros or None) in the interchange form."""
    _need(packed, "packed", torch.uint8, "cpu")
    nb = w4a8_packed_bytes(N, K, group, zeros)
    # (Exactly these bytes, as for the products: more are those of another form.)
    if packed.numel() > nb:
        raise ValueError(f"packed must have {nb} elements, got {packed.numel()}")
    _w4_scale_type(scale_dtype)
    groups = -(-K // group)
    codes = torch.empty((N, -(-K // 2)), dtype=torch.uint8)
    scales = torch.empty((N, groups), dtype=scale_dtype)
    z = torch.empty((N, groups), dtype=torch.uint8) if zeros else None
    _check(lib().unpack_w4a8(_ptr(packed), packed.numel(), N, K, group, _ptr(codes), _ptr(scales),
                             _ptr(z)), "unpack_w4a8")
    return codes, scales, z


@functools.lru_cache(maxsize=4096)
def w4a8_workspace_bytes(M: int, N: int, K: int) -> int:
    """Workspace bytes of w4a8_gemm (not to be cleared): 0 for one row and for short K."""
    v = int(lib().w4a8_workspace_bytes(M, N, K))
    if v < 0:
        raise W2A8Error(2, "w4a8_gemm")
    return v


def _w4_gemm(w_packed, x, s_a, M, N, K, group, scale_dtype, zeros, yf, yb, dev, workspace, stream):
    nw, need, pws = w4a8_packed_bytes(N, K, group, zeros), w4a8_workspace_bytes(M, N, K), None
    px = _mx4_ptr(x, "x", dev, torch.int8, M * K, M * K)
    ps = _mx4_ptr(s_a, "s_a", dev, torch.float32, M, M)
    code = _w4_scale_type(scale_dtype)
    # (Exactly these bytes: with zero points or groups of their own they are another number.)
    pw = _mx4_ptr(w_packed, "w_packed", dev, torch.uint8, nw, nw)
    if need:
        if workspace is None:
            workspace = _mx4_empty(x, (need,), torch.uint8, stream)
        pws = _mx4_ptr(workspace, "workspace", dev, torch.uint8, need)
    st = lib().w4a8_gemm(pw, px, ps, M, N, K, group, code, int(bool(zeros)), yf, yb, pws, need,
                         _mx4_stream(stream, dev))
    if st:
        raise W2A8Error(st, "w4a8_gemm")


def w4a8_gemm(w_packed, x, s_a, M, N, K, group, scale_dtype=torch.float16, zeros=False, y_f32=None,
              y_bf16=None, workspace=None, stream=None):
    """Raw C-ABI call: int8 rows times 4-bit weights with group scales (outputs must be
    given; workspace: uint8, at least w4a8_workspace_bytes, made here if not given); returns
    nothing."""
    dev = _mx4_gpu(x, "x")
    yf, yb = _mx4_outputs(y_f32, y_bf16, dev, M * N)
    _w4_gemm(w_packed, x, s_a, M, N, K, group, scale_dtype, zeros, yf, yb, dev, workspace, stream)


def gemm_w4a8(w_packed, x_q, s_a, N, K, group, scale_dtype=torch.float16, zeros=False,
              out_dtype=torch.float32, stream=None):
    """int8 rows x_q [M, K] (or [K]: one row) of scales s_a [M] times 4-bit weights with group
    scales -> fp32 or bf16 [M, N], M <= 64.  scale_dtype and zeros: of the packed weights."""
    dev = _mx4_gpu(x_q, "x_q")
    M, k = _mx4_rows(x_q, "x_q")
    if k != K:
        raise ValueError(f"x_q must have rows of {K} values, got {k}")
    y, yf, yb = _mx4_new(x_q, out_dtype, (M, N), stream)
    _w4_gemm(w_packed, x_q, s_a, M, N, K, group, scale_dtype, zeros, yf, yb, dev, None, stream)
    return y


def linear_w4a8(x_bf16, w_packed, N, K, group, scale_dtype=torch.float16, zeros=False,
                out_dtype=torch.float32, stream=None):
    """Linear layer with 4-bit weights: bf16 rows [M, K] (or [K]) -> fp32 or bf16 [M, N];
    quant_act_int8, then w4a8_gemm."""
    _mx4_gpu(x_bf16, "x_bf16")
    M, k = _mx4_rows(x_bf16, "x_bf16")
    if k != K:
        raise ValueError(f"x_bf16 must have rows of {K} values, got {k}")
    x_q, s_a = (_mx4_empty(x_bf16, (M, K), torch.int8, stream),
                _mx4_empty(x_bf16, (M,), torch.float32, stream))
    quant_act_int8(x_bf16, x_q, s_a, stream=stream)
    return gemm_w4a8(w_packed, x_q, s_a, N, K, group, scale_dtype, zeros, out_dtype, stream)


_ACTIVATIONS = {"silu": 0, "relu2": 1}


@functools.lru_cache(maxsize=4096)
def _moe_sizes(M, H, I, E, top_k):
    """Bytes of the workspace and of an expert's w_gate (or w_up) and w_down."""
    ws = int(lib().w2a8_moe_workspace_bytes(M, H, I, E, top_k))
    if ws < 0:
        raise W2A8Error(2, "w2a8_moe")
    return ws, packed_bytes(I, H), packed_bytes(H, I)


def w2a8_moe_workspace_bytes(M: int, H: int, I: int, E: int, top_k: int) -> int:
    """Workspace bytes of w2a8_moe (not to be cleared)."""
    return _moe_sizes(M, H, I, E, top_k)[0]


def _moe(x, s_a, logits, w_gate, w_up, w_down, s_gate, s_up, s_down, M, H, I, E, top_k, activation,
         renormalize, yf, yb, pws, ws_bytes, dev, stream):
    code = _mx4_type(logits, "logits")
    act = _ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be 'silu' or 'relu2', got {activation!r}")
    _, b1, b2 = _moe_sizes(M, H, I, E, top_k)
    u8, f32 = torch.uint8, torch.float32
    # (One expression for what fits; the checks one by one only say what does not: nine
    # calls of _mx4_ptr take 3.4 us of the host.)
    try:
        fits = (x.dtype is torch.int8 and x.get_device() == dev and x.is_contiguous() and x.numel() == M * H
                and s_a.dtype is f32 and s_a.get_device() == dev and s_a.is_contiguous() and s_a.numel() == M
                and logits.get_device() == dev and logits.numel() == M * E
                and w_gate.dtype is u8 and w_gate.get_device() == dev and w_gate.is_contiguous()
                and w_gate.numel() == E * b1
                and w_up.dtype is u8 and w_up.get_device() == dev and w_up.is_contiguous()
                and w_up.numel() == E * b1
                and w_down.dtype is u8 and w_down.get_device() == dev and w_down.is_contiguous()
                and w_down.numel() == E * b2
                and s_gate.dtype is f32 and s_gate.get_device() == dev and s_gate.is_contiguous()
                and s_gate.numel() == E
                and s_up.dtype is f32 and s_up.get_device() == dev and s_up.is_contiguous() and s_up.numel() == E
                and s_down.dtype is f32 and s_down.get_device() == dev and s_down.is_contiguous()
                and s_down.numel() == E)
    except AttributeError:
        fits = False
    if not fits:
        for t, name, dtype, n in ((x, "x", torch.int8, M * H), (s_a, "s_a", f32, M),
                                  (logits, "logits", logits.dtype, M * E), (w_gate, "w_gate", u8, E * b1),
                                  (w_up, "w_up", u8, E * b1), (w_down, "w_down", u8, E * b2),
                                  (s_gate, "s_gate", f32, E), (s_up, "s_up", f32, E), (s_down, "s_down", f32, E)):
            _mx4_ptr(t, name, dev, dtype, n, n)
        raise TypeError("the tensors of a mixture must be torch tensors")
    st = lib().w2a8_moe(
        x.data_ptr(), s_a.data_ptr(), logits.data_ptr(), code, w_gate.data_ptr(), w_up.data_ptr(),
        w_down.data_ptr(), s_gate.data_ptr(), s_up.data_ptr(), s_down.data_ptr(),
        M, H, I, E, top_k, act, int(bool(renormalize)), yf, yb, pws, ws_bytes, _mx4_stream(stream, dev))
    if st:
        raise W2A8Error(st, "w2a8_moe")


def w2a8_moe(x, s_a, logits, w_gate, w_up, w_down, s_gate, s_up, s_down, M, H, I, E, top_k,
             activation="silu", renormalize=True, y_f32=None, y_bf16=None, workspace=None,
             stream=None):
    """Raw C-ABI call (outputs must be given; workspace: uint8, at least
    w2a8_moe_workspace_bytes, made here if not given); returns nothing."""
    dev = _mx4_gpu(x, "x")
    yf, yb = _mx4_outputs(y_f32, y_bf16, dev, M * H)
    need = _moe_sizes(M, H, I, E, top_k)[0]
    if workspace is None:
        workspace = _mx4_empty(x, (need,), torch.uint8, stream)
    _moe(x, s_a, logits, w_gate, w_up, w_down, s_gate, s_up, s_down, M, H, I, E, top_k, activation,
         renormalize, yf, yb, _mx4_ptr(workspace, "workspace", dev, torch.uint8, need),
         workspace.numel(), dev, stream)


def moe(x_q, s_a, logits, w_gate, w_up, w_down, s_gate, s_up, s_down, H, I, top_k,
        activation="silu", renormalize=True, out_dtype=torch.float32, stream=None):
    """Mixture of ternary experts: int8 rows x_q [M, H] (or [H]: one row) of scales s_a [M] and
    router logits [M, E] (fp32, bf16 or fp16) -> fp32 or bf16 [M, H], M <= 64.

    w_gate, w_up: uint8 [E, packed_bytes(I, H)], w_down: uint8 [E, packed_bytes(H, I)], an
    expert a row (pack_ternary); s_gate, s_up, s_down: fp32 [E].  activation: "silu" or
    "relu2" (squared ReLU).  renormalize: the top_k experts' weights add up to one."""
    dev = _mx4_gpu(x_q, "x_q")
    M, k = _mx4_rows(x_q, "x_q")
    if k != H:
        raise ValueError(f"x_q must have rows of {H} values, got {k}")
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits must be a torch.Tensor")
    E = _mx4_rows(logits, "logits")[1]
    need = _moe_sizes(M, H, I, E, top_k)[0]
    y, yf, yb = _mx4_new(x_q, out_dtype, (M, H), stream)
    ws = _mx4_empty(x_q, (need,), torch.uint8, stream)
    _moe(x_q, s_a, logits, w_gate, w_up, w_down, s_gate, s_up, s_down, M, H, I, E, top_k, activation,
         renormalize, yf, yb, ws.data_ptr(), need, dev, stream)
    return y


# ---------------------------------------------------------------------------
# tuning knobs (w2a8_tuning.h)
# ---------------------------------------------------------------------------
DEFAULT_GEMV_POLICY = (4, 6, 8, 256, 48)


def tune_gemv(wg_per_cu: int, tiles_per_wave: int, unroll: int, krange_tiles: int = 256,
              split_min_tiles: int = 48):
    _check(lib().w2a8_tune_gemv(wg_per_cu, tiles_per_wave, unroll, krange_tiles,
                                split_min_tiles), "w2a8_tune_gemv")


def tune_gemv_force(kernel: int, waves_per_wg: int = 1, wgs_per_strip: int = 1, depth: int = 2,
                    direct_x: int = 0):
    """Force a GEMV plan (kernel 1: batch kernel, 2: ring kernel, 3: row-slice
    kernel with waves_per_wg 1 and wgs_per_strip 8; 0: automatic)."""
    _check(lib().w2a8_tune_gemv_force(kernel, waves_per_wg, wgs_per_strip, depth, direct_x),
           "w2a8_tune_gemv_force")


def tune_gemm(kernel: int):
    """Batched-product kernel: 0 automatic, 1 pipelined whenever K allows, 2 general,
    3 few-row whenever M <= 8, 4 short-batch MFMA ring whenever M <= 32 and K allows."""
    _check(lib().w2a8_tune_gemm(kernel), "w2a8_tune_gemm")


def tune_gemm_pipe(config: int = -1):
    """Forced configuration (0..9) of the pipelined MFMA GEMM (-1: automatic)."""
    _check(lib().w2a8_tune_gemm_pipe(config), "w2a8_tune_gemm_pipe")


def tune_gemm_ring(waves_per_wg: int = 0, wgs_per_strip: int = 0, depth: int = 0):
    """Forced plan of the short-batch MFMA ring kernel (all 0: automatic)."""
    _check(lib().w2a8_tune_gemm_ring(waves_per_wg, wgs_per_strip, depth), "w2a8_tune_gemm_ring")


def linear_plan(N: int, K: int, cus: int, int4: bool = False):
    """Automatic launch plan of the fused linear layer (w2a8_linear_gemv, or
    w2a4_linear_gemv with int4=True): (kernel, waves per workgroup,
    workgroups per strip, run, depth); kernel 1 is the workgroup kernel's
    fused variant, 3 the ring kernel over shared k-ranges, 4 the ring kernel
    with per-wave runs."""
    v = [ctypes.c_int(0) for _ in range(5)]
    _check(lib().w2a8_linear_plan(N, K, cus, int(bool(int4)), *[ctypes.byref(x) for x in v]),
           "w2a8_linear_plan")
    return tuple(x.value for x in v)


def mx4_plan(M: int, N: int, K: int, cus: int, ternary: bool = False, f32: bool = True,
             bf16: bool = False):
    """What gemm_w4mx4 (or gemm_w2mx4) runs for (M, N, K) on `cus` compute units into an fp32
    and/or a bf16 output: (kernel, rows, cols, groups, pass), see w2a8_tuning.h."""
    v = [ctypes.c_int() for _ in range(5)]
    _check(lib().w2a8_mx4_plan(M, N, K, int(bool(ternary)), int(bool(f32)) + 2 * int(bool(bf16)), cus,
                               *[ctypes.byref(x) for x in v]), "w2a8_mx4_plan")
    return tuple(x.value for x in v)


def w4a8_plan(M: int, N: int, K: int, group: int, cus: int):
    """What gemm_w4a8 runs for (M, N, K) and groups of `group` on `cus` compute units: (kernel, rows, groups, parts),
    see w2a8_tuning.h."""
    v = [ctypes.c_int() for _ in range(4)]
    _check(lib().w2a8_w4a8_plan(M, N, K, group, cus, *[ctypes.byref(x) for x in v]), "w2a8_w4a8_plan")
    return tuple(x.value for x in v)


def moe_plan(M: int, H: int, I: int, E: int, top_k: int, cus: int):
    """What moe runs for these sizes on `cus` compute units: (kernel, up, down), see
    w2a8_tuning.h."""
    v = [ctypes.c_int() for _ in range(3)]
    _check(lib().w2a8_moe_plan(M, H, I, E, top_k, cus, *[ctypes.byref(x) for x in v]),
           "w2a8_moe_plan")
    return tuple(x.value for x in v)


def tune_moe(kernel: int = 0):
    """Kernels of moe: 0 automatic, 1 one token at a time where its hidden rows fit LDS, 2 token
    rows together, 3 and 4 together with one and two strips to a workgroup."""
    _check(lib().w2a8_tune_moe(kernel), "w2a8_tune_moe")


def gemv_plan(N: int, K: int, cus: int):
    """Automatic launch plan of w2a8_gemv: (kernel, waves per workgroup,
    workgroups per strip, depth); kernel 2 is the ring kernel (K a multiple
    of 16), 1 the batch kernel."""
    kern, wk, sg, d = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
    _check(lib().w2a8_gemv_plan(N, K, cus, ctypes.byref(kern), ctypes.byref(wk), ctypes.byref(sg),
                                ctypes.byref(d)), "w2a8_gemv_plan")
    return kern.value, wk.value, sg.value, d.value
