"""Python binding of the sm_100a structured-sparse GEMM library (``libspgemm.so``).

Argument marshalling only: every function forwards torch tensors' device
pointers, sizes and the current CUDA stream to the C entry point of the same
name declared in ``include/spgemm.h``, and raises ``SpgError`` on a non-OK
status.  There is no fallback: if the shared library is missing or does not
load, importing the functions raises.  Build it with
``python -m structured_sparse_gemm_02_b200.build``.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libspgemm.so")

SPG_F16, SPG_BF16, SPG_S8, SPG_F32 = 0, 1, 2, 3
SPG_OUT_F16, SPG_OUT_S32 = 0, 1
SPG_X_MK, SPG_X_KM = 0, 1
SPG_ACT_NONE, SPG_ACT_GELU = 0, 1

_STATUS = {
    0: "SPG_OK", 1: "SPG_ERR_INVALID_ARG", 2: "SPG_ERR_UNSUPPORTED_SHAPE", 3: "SPG_ERR_MISALIGNED",
    4: "SPG_ERR_UNSUPPORTED_DEVICE", 5: "SPG_ERR_CUDA", 6: "SPG_ERR_TIMEOUT",
}

# Every exported symbol with its (restype, argtypes).
_i64, _i32, _p, _sz = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t


class SpgTwSizes(ctypes.Structure):
    _fields_ = [("N", _i64), ("K", _i64), ("Nk", _i64), ("G", _i32), ("T", _i32),
                ("offsetk_len", _i64), ("wc_elems", _i64), ("reorg_ws_bytes", _i64)]


class SpgTwDesc(ctypes.Structure):
    _fields_ = [("N", _i64), ("K", _i64), ("Nk", _i64), ("G", _i32), ("T", _i32),
                ("offsetk_len", _i64), ("offsetn", _p), ("tile_n0", _p), ("tile_kofs", _p),
                ("k_per_tile", _p), ("offsetk", _p), ("Wc", _p)]


SIGNATURES = {
    "spg_version": (ctypes.c_int, []),
    "spg_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "spg_check_device_error": (ctypes.c_int, [_p, ctypes.POINTER(ctypes.c_uint32)]),
    "spg_selftest_bounded_wait": (ctypes.c_int, [_i64, _p]),
    "sparse_prune_24": (ctypes.c_int, [_p, _i64, _p, _i64, _i64, _i64, ctypes.c_int, _p]),
    "sparse_compress_24": (ctypes.c_int, [_p, _i64, _p, _p, _i64, _i64, ctypes.c_int, _p]),
    "spgemm_24_f16": (ctypes.c_int, [_p, _i64, _p, _p, _p, _p, _i64, _i64, _i64, _i64, ctypes.c_int, _p]),
    "spgemm_24_f16_host": (ctypes.c_int, [_p, _i64, _p, _p, _p, _p, _i64, _i64, _i64, _i64, ctypes.c_int, _p, _p,
                                          _i64, _p]),
    "spgemm_24_f16_gelu": (ctypes.c_int, [_p, _i64, _p, _p, _p, _p, _i64, _i64, _i64, _i64, ctypes.c_int, _p]),
    "spgemm_24_f16_yt": (ctypes.c_int, [_p, _i64, _p, _p, _p, _p, _i64, _i64, _i64, _i64, ctypes.c_int, _p]),
    "spgemm_24_s8": (ctypes.c_int, [_p, _i64, _p, _p, _p, _p, _p, _i64, ctypes.c_int, _i64, _i64, _i64, _p]),
    "spgemm_24_s8_q": (ctypes.c_int, [_p, _i64, _p, _p, _p, _p, ctypes.c_float, ctypes.c_int, _p, _i64, _i64, _i64,
                                      _i64, _p]),
    "tw_query_sizes": (ctypes.c_int, [_i64, _i64, _i32, _i64, ctypes.POINTER(_i32), ctypes.POINTER(SpgTwSizes)]),
    "tw_reorganize": (ctypes.c_int, [_p, _i64, _i64, ctypes.POINTER(_i32), ctypes.POINTER(SpgTwDesc), _p, _sz,
                                     _p]),
    "tw_workspace_size": (_sz, [_i64, _i64, ctypes.c_int]),
    "spgemm_tw_f16": (ctypes.c_int, [_p, _i64, ctypes.c_int, ctypes.POINTER(SpgTwDesc), _p, _i64, _i64, _p,
                                     _sz, _p]),
    "spgemm_tw_f16_yt": (ctypes.c_int, [_p, _i64, ctypes.c_int, ctypes.POINTER(SpgTwDesc), _p, _i64, _i64, _p,
                                        _sz, _p]),
    "tw_condense_f32": (ctypes.c_int, [_p, _i64, ctypes.POINTER(SpgTwDesc), _p, _p]),
    "tw_workspace_size_f32": (_sz, [_i64, _i64, ctypes.c_int]),
    "spgemm_tw_f32": (ctypes.c_int, [_p, _i64, ctypes.c_int, ctypes.POINTER(SpgTwDesc), _p, _p, _i64, _i64, _p, _sz,
                                     _p]),
    "spgemm_tw_f16_noalloc": (ctypes.c_int, [_p, _i64, ctypes.POINTER(SpgTwDesc), _p, _i64, _i64, _p]),
    "lora_plan_size": (_sz, [_i64, _i64]),
    "lora_plan": (ctypes.c_int, [_p, _i64, _i64, _p, _sz, _p]),
    "lora_f16": (ctypes.c_int, [_p, _i64, _p, _p, _p, _p, _p, _i64, _p, _i64, _p, _i64, _i64, _i64, _i64, _i64, _i64,
                                ctypes.c_int, _p]),
    "lora_bwd_workspace_size": (_sz, [_i64, _i64, _i64, _i64, _i64]),
    "lora_f16_bwd": (ctypes.c_int, [_p, _i64, _p, _i64, _p, _i64, _p, _p, _p, _p, _p, _i64, _p, _i64, _p, _p, _p, _sz,
                                    _i64, _i64, _i64, _i64, _i64, ctypes.c_int, _p]),
    "layernorm": (ctypes.c_int, [_p, _i64, _p, _i64, _p, _i64, _p, _p, ctypes.c_float, _p, _i64, _p, _p, _i64, _i64,
                                 ctypes.c_int, ctypes.c_int, _p]),
    "layernorm_s8": (ctypes.c_int, [_p, _i64, _p, _i64, _p, _i64, _p, _p, ctypes.c_float, ctypes.c_float, _p, _i64,
                                    _i64, _i64, ctypes.c_int, ctypes.c_int, _p]),
    "layernorm_bwd_workspace_size": (_sz, [_i64, _i64, ctypes.c_int]),
    "layernorm_bwd": (ctypes.c_int, [_p, _i64, _p, _i64, _p, _p, _p, _p, _i64, _p, _i64, _p, _p, _p, _sz, _i64, _i64,
                                     ctypes.c_int, ctypes.c_int, _p]),
}

_lib = None


class SpgError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {_STATUS.get(status, status)}")
        self.status = status


def lib() -> ctypes.CDLL:
    """The loaded shared library (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m structured_sparse_gemm_02_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


_torch = None
_FLOAT_CODES: dict = {}
_device = None  # the current device's index
_raw = None     # a device's current stream without a Stream object (3 us), where torch offers that


def _tm():
    """torch, imported with the first call that needs it (the package itself also builds without it)."""
    global _torch, _device, _raw
    if _torch is None:
        import torch
        _device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        _raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _FLOAT_CODES.update({torch.float16: SPG_F16, torch.bfloat16: SPG_BF16, torch.float32: SPG_F32})
        _torch = torch
    return _torch


def _check(fn: str, st: int) -> None:
    if st != 0:
        raise SpgError(fn, st)


def _stream(stream) -> int:
    if stream is None:
        if _raw is not None:
            return _raw(_device())
        stream = _tm().cuda.current_stream()
    return int(getattr(stream, "cuda_stream", stream))


def _dtype_code(t) -> int:
    import torch
    return {torch.float16: SPG_F16, torch.bfloat16: SPG_BF16, torch.int8: SPG_S8}[t.dtype]


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _on_device(t, name: str) -> None:
    """A tensor whose pointer goes to a kernel lives on the current CUDA device."""
    torch = _tm()
    if t.is_cuda and t.get_device() == _device():
        return
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor (it is on {t.device})")
    raise ValueError(f"{name} is on {t.device}, the current device is cuda:{torch.cuda.current_device()}")


def _arg(t, name: str, dtypes, shape=None, contiguous=False, optional=False):
    """Check a tensor argument before its pointer reaches the library: dtype, exact
    shape, row-major layout with unit column stride (the C ABI passes only the
    row pitch), contiguity where the ABI fixes the pitch, and the device.
    Returns t (None is accepted only for optional arguments)."""
    import torch
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype}, expected one of {tuple(dtypes)}")
    if shape is not None and tuple(t.shape) != tuple(int(v) for v in shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(int(v) for v in shape)}")
    if t.dim() == 2 and t.numel() > 0 and t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must be row-major with unit column stride (got strides {t.stride()})")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    _on_device(t, name)
    return t


def _nbytes(t) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def _types(*names):
    import torch
    return tuple(getattr(torch, n) for n in names)


def version() -> int:
    return lib().spg_version()


def check_device_error(stream=None) -> int:
    """Synchronise ``stream`` and return the device error bits (0 = none)."""
    bits = ctypes.c_uint32(0)
    st = lib().spg_check_device_error(_stream(stream), ctypes.byref(bits))
    if st not in (0, 6):
        _check("spg_check_device_error", st)
    return int(bits.value)


def selftest_bounded_wait(limit_ns: int = 20_000_000, stream=None) -> None:
    """Launch the self-test whose bounded wait runs out (see spgemm.h); read the
    result with check_device_error()."""
    _check("spg_selftest_bounded_wait", lib().spg_selftest_bounded_wait(int(limit_ns), _stream(stream)))


def sparse_prune_24(W, Wm=None, stream=None):
    """2:4 magnitude prune of W [N, K] (row pitch = W.stride(0)); returns Wm."""
    import torch
    _arg(W, "W", _types("float16", "bfloat16", "int8"))
    N, K = W.shape
    if Wm is None:
        Wm = torch.empty_like(W)
    _arg(Wm, "Wm", (W.dtype,), (N, K))
    _check("sparse_prune_24", lib().sparse_prune_24(
        _ptr(W), W.stride(0), _ptr(Wm), Wm.stride(0), N, K, _dtype_code(W), _stream(stream)))
    return Wm


def sparse_compress_24(W, Wv=None, meta=None, stream=None):
    """2:4 compress W [N, K] into (Wv [N, K/2], meta uint8 [N, K/8])."""
    import torch
    _arg(W, "W", _types("float16", "bfloat16", "int8"))
    N, K = W.shape
    if Wv is None:
        Wv = torch.empty((N, K // 2), dtype=W.dtype, device=W.device)
    if meta is None:
        meta = torch.empty((N, K // 8), dtype=torch.uint8, device=W.device)
    _arg(Wv, "Wv", (W.dtype,), (N, K // 2), contiguous=True)
    _arg(meta, "meta", _types("uint8"), (N, K // 8), contiguous=True)
    _check("sparse_compress_24", lib().sparse_compress_24(
        _ptr(W), W.stride(0), _ptr(Wv), _ptr(meta), N, K, _dtype_code(W), _stream(stream)))
    return Wv, meta


def _check_24(X, Wv, meta, dtypes):
    """X [M, K], Wv [N, K/2] (same dtype, contiguous), meta [N, K/8] uint8 (contiguous); returns M, K, N."""
    _arg(X, "X", dtypes)
    if X.dim() != 2 or Wv is None or Wv.dim() != 2:
        raise ValueError("X and Wv must be 2-D")
    M, K = X.shape
    N = Wv.shape[0]
    _arg(Wv, "Wv", (X.dtype,), (N, K // 2), contiguous=True)
    _arg(meta, "meta", _types("uint8"), (N, K // 8), contiguous=True)
    return M, K, N


def spgemm_24_f16(X, Wv, meta, bias=None, Y=None, stream=None):
    """Y [M, N] = X [M, K] . decompress(Wv, meta)^T (+ bias), fp16 or bf16."""
    import torch
    M, K, N = _check_24(X, Wv, meta, _types("float16", "bfloat16"))
    _arg(bias, "bias", (X.dtype,), (N,), contiguous=True, optional=True)
    if Y is None:
        Y = torch.empty((M, N), dtype=X.dtype, device=X.device)
    _arg(Y, "Y", (X.dtype,), (M, N))
    _check("spgemm_24_f16", lib().spgemm_24_f16(
        _ptr(X), X.stride(0), _ptr(Wv), _ptr(meta), _ptr(bias), _ptr(Y), Y.stride(0), M, N, K,
        _dtype_code(X), _stream(stream)))
    return Y


def _host_arg(t, name: str, dtypes, shape) -> None:
    """A host tensor whose pointer goes to a host <-> device copy: dtype, shape,
    row-major with unit column stride, in CPU memory."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cpu":
        raise ValueError(f"{name} must be in host memory (it is on {t.device})")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype}, expected one of {tuple(dtypes)}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dim() == 2 and t.numel() > 0 and t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must be row-major with unit column stride")


def spgemm_24_f16_host(X_host, Wv, meta, bias, Y_host, X_dev, Y_dev, stream=None):
    """spgemm_24_f16 from and to host memory (page-locked for asynchronous
    copies): X_host [M, K] -> X_dev [M, K] (contiguous), the layer into Y_dev
    [M, N], Y_dev -> Y_host [M, N], all queued on the stream."""
    dts = _types("float16", "bfloat16")
    _arg(X_dev, "X_dev", dts, contiguous=True)
    M, K, N = _check_24(X_dev, Wv, meta, dts)
    _host_arg(X_host, "X_host", (X_dev.dtype,), (M, K))
    _host_arg(Y_host, "Y_host", (X_dev.dtype,), (M, N))
    _arg(bias, "bias", (X_dev.dtype,), (N,), contiguous=True, optional=True)
    _arg(Y_dev, "Y_dev", (X_dev.dtype,), (M, N))
    _check("spgemm_24_f16_host", lib().spgemm_24_f16_host(
        _ptr(X_host), X_host.stride(0), _ptr(Wv), _ptr(meta), _ptr(bias), _ptr(Y_host), Y_host.stride(0), M, N, K,
        _dtype_code(X_dev), _ptr(X_dev), _ptr(Y_dev), Y_dev.stride(0), _stream(stream)))
    return Y_host


def spgemm_24_f16_gelu(X, Wv, meta, bias=None, Y=None, stream=None):
    """Y [M, N] = GELU(X [M, K] . decompress(Wv, meta)^T (+ bias)), fp16 or bf16."""
    import torch
    M, K, N = _check_24(X, Wv, meta, _types("float16", "bfloat16"))
    _arg(bias, "bias", (X.dtype,), (N,), contiguous=True, optional=True)
    if Y is None:
        Y = torch.empty((M, N), dtype=X.dtype, device=X.device)
    _arg(Y, "Y", (X.dtype,), (M, N))
    _check("spgemm_24_f16_gelu", lib().spgemm_24_f16_gelu(
        _ptr(X), X.stride(0), _ptr(Wv), _ptr(meta), _ptr(bias), _ptr(Y), Y.stride(0), M, N, K,
        _dtype_code(X), _stream(stream)))
    return Y


def spgemm_24_f16_yt(X, Wv, meta, bias=None, Yt=None, stream=None):
    """Yt [N, M] = (X [M, K] . decompress(Wv, meta)^T (+ bias))^T, fp16 or bf16."""
    import torch
    M, K, N = _check_24(X, Wv, meta, _types("float16", "bfloat16"))
    _arg(bias, "bias", (X.dtype,), (N,), contiguous=True, optional=True)
    if Yt is None:
        Yt = torch.empty((N, M), dtype=X.dtype, device=X.device)
    _arg(Yt, "Yt", (X.dtype,), (N, M))
    _check("spgemm_24_f16_yt", lib().spgemm_24_f16_yt(
        _ptr(X), X.stride(0), _ptr(Wv), _ptr(meta), _ptr(bias), _ptr(Yt), Yt.stride(0), M, N, K,
        _dtype_code(X), _stream(stream)))
    return Yt


def spgemm_24_s8(X, Wv, meta, scale=None, bias=None, Y=None, out_mode=SPG_OUT_F16, stream=None):
    """int8 2:4 GEMM; out_mode SPG_OUT_F16 (dequantised fp16) or SPG_OUT_S32 (raw int32)."""
    import torch
    M, K, N = _check_24(X, Wv, meta, _types("int8"))
    _arg(scale, "scale", _types("float32"), (N,), contiguous=True, optional=out_mode == SPG_OUT_S32)
    _arg(bias, "bias", _types("float16"), (N,), contiguous=True, optional=True)
    ydt = torch.int32 if out_mode == SPG_OUT_S32 else torch.float16
    if Y is None:
        Y = torch.empty((M, N), dtype=ydt, device=X.device)
    _arg(Y, "Y", (ydt,), (M, N))
    _check("spgemm_24_s8", lib().spgemm_24_s8(
        _ptr(X), X.stride(0), _ptr(Wv), _ptr(meta), _ptr(scale), _ptr(bias), _ptr(Y), Y.stride(0),
        out_mode, M, N, K, _stream(stream)))
    return Y


def spgemm_24_s8_q(X, Wv, meta, scale, bias=None, qscale=1.0, act=SPG_ACT_NONE, Yq=None, stream=None):
    """int8 2:4 layer whose epilogue emits int8 activations for the next int8 layer:
    Yq = clamp(rne(act(fp32(acc) * scale (+ bias)) * qscale), -127, 127)."""
    import torch
    M, K, N = _check_24(X, Wv, meta, _types("int8"))
    _arg(scale, "scale", _types("float32"), (N,), contiguous=True)
    _arg(bias, "bias", _types("float16"), (N,), contiguous=True, optional=True)
    if Yq is None:
        Yq = torch.empty((M, N), dtype=torch.int8, device=X.device)
    _arg(Yq, "Yq", _types("int8"), (M, N))
    _check("spgemm_24_s8_q", lib().spgemm_24_s8_q(
        _ptr(X), X.stride(0), _ptr(Wv), _ptr(meta), _ptr(scale), _ptr(bias), float(qscale), int(act), _ptr(Yq),
        Yq.stride(0), M, N, K, _stream(stream)))
    return Yq


class TwDesc:
    """Device buffers of a tile-wise descriptor (see ``spg_tw_desc`` in include/spgemm.h)."""

    def __init__(self, N: int, K: int, G: int, n_pruned: int, k_per_tile: Sequence[int], device="cuda"):
        import torch
        kpt = (ctypes.c_int32 * len(k_per_tile))(*[int(v) for v in k_per_tile])
        sz = SpgTwSizes()
        _check("tw_query_sizes", lib().tw_query_sizes(N, K, G, n_pruned, kpt, ctypes.byref(sz)))
        self.sizes = sz
        self.k_host = kpt
        self.n_pruned = n_pruned
        i32 = dict(dtype=torch.int32, device=device)
        self.offsetn = torch.empty(sz.Nk, **i32)
        self.tile_n0 = torch.empty(sz.T + 1, **i32)
        self.tile_kofs = torch.empty(sz.T + 1, **i32)
        self.k_per_tile = torch.empty(sz.T, **i32)
        self.offsetk = torch.empty(max(1, sz.offsetk_len), **i32)
        self.Wc = torch.empty(max(1, sz.wc_elems), dtype=torch.float16, device=device)
        self.c = SpgTwDesc(sz.N, sz.K, sz.Nk, sz.G, sz.T, sz.offsetk_len, self.offsetn.data_ptr(),
                           self.tile_n0.data_ptr(), self.tile_kofs.data_ptr(), self.k_per_tile.data_ptr(),
                           self.offsetk.data_ptr(), self.Wc.data_ptr())


def tw_reorganize(W, G: int, n_pruned: int, k_per_tile: Sequence[int], workspace=None, stream=None) -> TwDesc:
    """Condense a dense fp16 W [N, K] into a tile-wise descriptor."""
    import torch
    _arg(W, "W", _types("float16"))
    N, K = W.shape
    d = TwDesc(N, K, G, n_pruned, k_per_tile, device=W.device)
    if workspace is None:
        workspace = torch.empty(max(16, d.sizes.reorg_ws_bytes), dtype=torch.uint8, device=W.device)
    _arg(workspace, "workspace", (workspace.dtype,), contiguous=True)
    _check("tw_reorganize", lib().tw_reorganize(_ptr(W), W.stride(0), n_pruned, d.k_host, ctypes.byref(d.c),
                                                _ptr(workspace), _nbytes(workspace), _stream(stream)))
    return d


def _check_tw_x(X, desc, x_layout, M, dtypes):
    """X is [M, K] (SPG_X_MK) or [K, M] (SPG_X_KM) with K the descriptor's; returns M."""
    if x_layout not in (SPG_X_MK, SPG_X_KM):
        raise ValueError(f"x_layout must be SPG_X_MK or SPG_X_KM, not {x_layout}")
    _arg(X, "X", dtypes)
    if X.dim() != 2:
        raise ValueError("X must be 2-D")
    if M is None:
        M = X.shape[0] if x_layout == SPG_X_MK else X.shape[1]
    K = desc.sizes.K
    want = (M, K) if x_layout == SPG_X_MK else (K, M)
    if tuple(X.shape) != want:
        raise ValueError(f"X: shape {tuple(X.shape)}, expected {want} for this layout and descriptor")
    return int(M)


def _workspace(workspace, need: int, device):
    """The caller's workspace (checked against the size the call needs) or a new one."""
    import torch
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=device) if need else None
    _arg(workspace, "workspace", (workspace.dtype,), contiguous=True)
    if _nbytes(workspace) < need:
        raise ValueError(f"workspace holds {_nbytes(workspace)} bytes, the call needs {need}")
    return workspace


def tw_workspace_size(M: int, K: int, x_layout: int) -> int:
    return int(lib().tw_workspace_size(M, K, x_layout))


def spgemm_tw_f16(X, desc: TwDesc, x_layout=SPG_X_MK, Y=None, workspace=None, M: Optional[int] = None,
                  stream=None):
    """Tile-wise GEMM: X [M, K] (SPG_X_MK) or [K, M] (SPG_X_KM) -> Y [M, N] fp16."""
    import torch
    M = _check_tw_x(X, desc, x_layout, M, _types("float16"))
    N = desc.sizes.N
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.float16, device=X.device)
    _arg(Y, "Y", _types("float16"), (M, N))
    workspace = _workspace(workspace, tw_workspace_size(M, desc.sizes.K, x_layout), X.device)
    _check("spgemm_tw_f16", lib().spgemm_tw_f16(
        _ptr(X), X.stride(0), x_layout, ctypes.byref(desc.c), _ptr(Y), Y.stride(0), M, _ptr(workspace),
        _nbytes(workspace), _stream(stream)))
    return Y


def spgemm_tw_f16_yt(X, desc: TwDesc, x_layout=SPG_X_MK, Yt=None, workspace=None, M: Optional[int] = None,
                     stream=None):
    """Tile-wise GEMM writing Yt [N, M] = Y^T (the [K, M] activations of a following tile-wise layer)."""
    import torch
    M = _check_tw_x(X, desc, x_layout, M, _types("float16"))
    N = desc.sizes.N
    if Yt is None:  # rows of Yt padded to a multiple of 8 elements (the ABI's 16-byte pitch)
        Yt = torch.empty((N, (M + 7) // 8 * 8), dtype=torch.float16, device=X.device)[:, :M]
    _arg(Yt, "Yt", _types("float16"), (N, M))
    workspace = _workspace(workspace, tw_workspace_size(M, desc.sizes.K, x_layout), X.device)
    _check("spgemm_tw_f16_yt", lib().spgemm_tw_f16_yt(
        _ptr(X), X.stride(0), x_layout, ctypes.byref(desc.c), _ptr(Yt), Yt.stride(0), M, _ptr(workspace),
        _nbytes(workspace), _stream(stream)))
    return Yt


def tw_condense_f32(W, desc: TwDesc, Wc32=None, stream=None):
    """fp32 condensed tiles of W [N, K] (fp32) through the pattern of ``desc``."""
    import torch
    _arg(W, "W", _types("float32"), (desc.sizes.N, desc.sizes.K))
    if Wc32 is None:
        Wc32 = torch.empty(desc.sizes.wc_elems, dtype=torch.float32, device=W.device)
    _arg(Wc32, "Wc32", _types("float32"), contiguous=True)
    if Wc32.numel() < desc.sizes.wc_elems:
        raise ValueError(f"Wc32 holds {Wc32.numel()} elements, the descriptor needs {desc.sizes.wc_elems}")
    _check("tw_condense_f32", lib().tw_condense_f32(_ptr(W), W.stride(0), ctypes.byref(desc.c), _ptr(Wc32),
                                                    _stream(stream)))
    return Wc32


def spgemm_tw_f32(X, desc: TwDesc, Wc32, x_layout=SPG_X_MK, Y=None, workspace=None, M: Optional[int] = None,
                  stream=None):
    """Tile-wise GEMM in fp32 on the CUDA cores: X [M, K] or [K, M] -> Y [M, N] fp32."""
    import torch
    M = _check_tw_x(X, desc, x_layout, M, _types("float32"))
    N = desc.sizes.N
    _arg(Wc32, "Wc32", _types("float32"), contiguous=True)
    if Wc32.numel() < desc.sizes.wc_elems:
        raise ValueError(f"Wc32 holds {Wc32.numel()} elements, the descriptor needs {desc.sizes.wc_elems}")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.float32, device=X.device)
    _arg(Y, "Y", _types("float32"), (M, N))
    workspace = _workspace(workspace, int(lib().tw_workspace_size_f32(M, desc.sizes.K, x_layout)), X.device)
    _check("spgemm_tw_f32", lib().spgemm_tw_f32(
        _ptr(X), X.stride(0), x_layout, ctypes.byref(desc.c), _ptr(Wc32), _ptr(Y), Y.stride(0), M, _ptr(workspace),
        _nbytes(workspace), _stream(stream)))
    return Y


def spgemm_tw_f16_noalloc(X, desc: TwDesc, Y=None, stream=None):
    """Tile-wise GEMM on X [M, K] for callers that cannot allocate device memory.

    The transposed activations live in the library's fixed 8 MiB device array
    (M * K * 2 bytes at most) instead of a workspace; calls sharing it must not
    overlap on the GPU.
    """
    import torch
    M = _check_tw_x(X, desc, SPG_X_MK, None, _types("float16"))
    N = desc.sizes.N
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.float16, device=X.device)
    _arg(Y, "Y", _types("float16"), (M, N))
    _check("spgemm_tw_f16_noalloc", lib().spgemm_tw_f16_noalloc(
        _ptr(X), X.stride(0), ctypes.byref(desc.c), _ptr(Y), Y.stride(0), M, _stream(stream)))
    return Y


def _like(t, name: str, dtype, shape, dev: int) -> int:
    """_arg for the further tensors of a call whose first one passed it (its device is
    ``dev``): a valid tensor costs a few comparisons, any other one gets _arg's message.
    Matrices may have a row pitch, which is returned; others are contiguous."""
    if t.__class__ is _torch.Tensor or isinstance(t, _torch.Tensor):
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev:
            if len(shape) == 2:
                ld, unit = t.stride()
                if unit == 1 or shape[1] <= 1 or not shape[0]:
                    # a single row has no pitch of its own: the next multiple of 16
                    return ld if shape[0] > 1 else (shape[1] + 15) // 16 * 16
            elif t.is_contiguous():
                return 0
    _arg(t, name, (dtype,), shape, contiguous=len(shape) != 2)
    raise ValueError(f"{name} is on {t.device}, the other arguments are on device {dev}")


def _first(t, name: str, dtypes, dims: int = 2) -> int:
    """_arg for a call's first tensor; returns its row pitch."""
    if not isinstance(t, _tm().Tensor) or t.dtype not in dtypes or t.dim() != dims:
        _arg(t, name, dtypes)
        raise ValueError(f"{name} must be {dims}-D")
    _on_device(t, name)
    if dims == 2:
        ld, unit = t.stride()
        M, C = t.shape
        if unit == 1 or C <= 1 or not M:
            return ld if M > 1 else (C + 15) // 16 * 16
    return _like(t, name, t.dtype, t.shape, t.get_device())


def _on_stream(stream, device):
    """The stream as a torch stream (a raw handle is wrapped)."""
    torch = _tm()
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)), device=device)


def _new(shape, dtype, like, stream, pad=False):
    """A tensor that the call writes, on the device of ``like``.  Where the call goes to
    another stream than the current one, the memory is that stream's, so that neither its
    last use nor its next one can overlap the call.  ``pad``: rows padded to 16 bytes."""
    if stream is not None and like.is_cuda:
        with _torch.cuda.stream(_on_stream(stream, like.device)):
            return _new(shape, dtype, like, None, pad)
    if shape == like.shape and dtype is like.dtype and like.is_contiguous() and not (
            pad and (shape[1] * dtype.itemsize) % 16) and (len(shape) != 2 or like.stride(0) >= shape[1]):
        return _torch.empty_like(like)  # the cheapest way to say the same (a single row may have any stride)
    if pad:
        M, C = shape
        step = 16 // dtype.itemsize
        if C % step:
            return like.new_empty((M, (C + step - 1) // step * step), dtype=dtype)[:, :C]
    return like.new_empty(shape, dtype=dtype)


def _apart(**outs) -> None:
    """The call's outputs do not share memory: each byte is written for one of them.  Their
    spans are compared, so columns of one buffer side by side are refused too."""
    spans = []
    for name, t in outs.items():
        if t is not None and t.numel():
            n = (t.shape[0] - 1) * t.stride(0) + t.shape[1] if t.dim() == 2 else t.numel()
            spans.append((t.data_ptr(), t.data_ptr() + n * t.element_size(), name))
    spans.sort()
    for (_, end, a), (start, _, b) in zip(spans, spans[1:]):
        if start < end:
            raise ValueError(f"{a} and {b} share memory, or rows of one lie between rows of the other")


def _ln_args(X, gamma):
    """X [M, C] and gamma [C] of the layer norm calls; returns X's pitch and device index and the type codes."""
    torch = _tm()
    ldx = _first(X, "X", (torch.float16, torch.bfloat16, torch.float32))
    dev = X.get_device()
    wdt = torch.float32 if getattr(gamma, "dtype", None) is torch.float32 else X.dtype
    _like(gamma, "gamma", wdt, X.shape[1:], dev)
    return ldx, dev, _FLOAT_CODES[X.dtype], _FLOAT_CODES[wdt]


def _ln_fwd(fn, X, gamma, beta, eps, qscale, residual, H, Y, ydt, stats, stream):
    ldx, dev, code, wcode = _ln_args(X, gamma)
    shape, dt = X.shape, X.dtype
    M, C = shape
    if beta is not None:
        _like(beta, "beta", gamma.dtype, gamma.shape, dev)
    res = h = None
    ldres = ldh = 0
    if residual is not None:
        ldres = _like(residual, "residual", dt, shape, dev)
        res = residual.data_ptr()
        if H is None:
            H = _new(shape, dt, X, stream, pad=True)
            ldh = H.stride(0)
        else:
            ldh = _like(H, "H", dt, shape, dev)
        h = H.data_ptr()
    elif H is not None:
        raise ValueError("H is the sum of X and residual: it needs a residual")
    if Y is None:
        Y = _new(shape, ydt, X, stream, pad=True)
        ldy = Y.stride(0)
    else:
        ldy = _like(Y, "Y", ydt, shape, dev)
        _apart(Y=Y, H=H)
    if qscale is None:
        mean = rstd = None
        if stats:
            mean = _new((M,), _torch.float32, X, stream)
            rstd = _new((M,), _torch.float32, mean, stream)
        _check(fn, lib().layernorm(
            X.data_ptr(), ldx, res, ldres, h, ldh, gamma.data_ptr(), _ptr(beta), eps, Y.data_ptr(), ldy, _ptr(mean),
            _ptr(rstd), M, C, code, wcode, _stream(stream)))
        return Y, H, mean, rstd
    _check(fn, lib().layernorm_s8(
        X.data_ptr(), ldx, res, ldres, h, ldh, gamma.data_ptr(), _ptr(beta), eps, qscale, Y.data_ptr(), ldy, M, C,
        code, wcode, _stream(stream)))
    return Y, H


def layernorm(X, gamma, beta=None, eps=1e-5, residual=None, H=None, Y=None, stats=False, stream=None):
    """Layer norm of X [M, C] (or of H = X + residual), fp16, bf16 or fp32; gamma and
    beta [C] in X's dtype or fp32.  Returns (Y, H, mean, rstd): H is None without a
    residual, mean and rstd (fp32 [M], for layernorm_bwd) are None without ``stats``.
    Outputs that the caller gives, here and in the calls below, take a stretch of memory each."""
    return _ln_fwd("layernorm", X, gamma, beta, eps, None, residual, H, Y, getattr(X, "dtype", None), stats, stream)


def layernorm_s8(X, gamma, beta, qscale, eps=1e-5, residual=None, H=None, Yq=None, stream=None):
    """Layer norm of X [M, C] (or of H = X + residual) quantised to the int8 activations of
    an int8 2:4 layer: Yq = clamp(rne(y * qscale), -127, 127).  Returns (Yq, H)."""
    return _ln_fwd("layernorm_s8", X, gamma, beta, eps, float(qscale), residual, H, Yq, _tm().int8, False, stream)


def layernorm_bwd(dY, X, mean, rstd, gamma, dH=None, dX=None, dgamma=None, dbeta=None, workspace=None, stream=None):
    """Gradients of layernorm: X is what the norm was taken of (H where there was a
    residual), dH [M, C] the gradient that reaches it by the residual path.  Returns
    (dX, dgamma, dbeta), the last two in gamma's dtype."""
    ldx, dev, code, wcode = _ln_args(X, gamma)
    shape, dt, wdt = X.shape, X.dtype, gamma.dtype
    M, C = shape
    lddy = _like(dY, "dY", dt, shape, dev)
    _like(mean, "mean", _torch.float32, (M,), dev)
    _like(rstd, "rstd", _torch.float32, (M,), dev)
    lddh = 0 if dH is None else _like(dH, "dH", dt, shape, dev)
    given = not (dX is None and dgamma is None and dbeta is None and workspace is None)
    if dX is None:
        dX = _new(shape, dt, X, stream, pad=True)
        lddx = dX.stride(0)
    else:
        lddx = _like(dX, "dX", dt, shape, dev)
    dgamma = _new((C,), wdt, gamma, stream) if dgamma is None else dgamma
    dbeta = _new((C,), wdt, gamma, stream) if dbeta is None else dbeta
    need = lib().layernorm_bwd_workspace_size(M, C, code)
    if workspace is None:
        workspace = _new((need,), _torch.uint8, X, stream)
    if given:
        _workspace(workspace, need, X.device)
        _like(dgamma, "dgamma", wdt, (C,), dev)
        _like(dbeta, "dbeta", wdt, (C,), dev)
        _apart(dX=dX, dgamma=dgamma, dbeta=dbeta, workspace=workspace)
    _check("layernorm_bwd", lib().layernorm_bwd(
        dY.data_ptr(), lddy, X.data_ptr(), ldx, mean.data_ptr(), rstd.data_ptr(), gamma.data_ptr(), _ptr(dH), lddh,
        dX.data_ptr(), lddx, dgamma.data_ptr(), dbeta.data_ptr(), workspace.data_ptr(), _nbytes(workspace), M, C, code,
        wcode, _stream(stream)))
    return dX, dgamma, dbeta


class LoraPlan:
    """The rows of a batch grouped by adapter (device memory filled by ``lora_plan``)."""

    def __init__(self, buf, M: int, L: int):
        self.buf, self.M, self.L = buf, M, L


def lora_plan(index, L: int, plan: Optional[LoraPlan] = None, stream=None) -> LoraPlan:
    """Group the rows of a batch by adapter: index int32 [M] names the adapter of each row,
    values outside [0, L) none.  One plan serves every layer's lora_f16 and
    lora_f16_bwd of the batch.  ``plan`` refills an earlier plan of the same M and L."""
    torch = _tm()
    _first(index, "index", (torch.int32,), dims=1)
    M, L = index.shape[0], int(L)
    need = lib().lora_plan_size(M, L)
    if plan is None:
        plan = LoraPlan(_new((need // 4,), torch.int32, index, stream), M, L)
    elif plan.M != M or plan.L != L:
        raise ValueError(f"plan is for {plan.M} rows and {plan.L} adapters, the index for {M} and {L}")
    else:
        _like(plan.buf, "plan", torch.int32, (need // 4,), index.get_device())
    _check("lora_plan", lib().lora_plan(index.data_ptr(), M, L, plan.buf.data_ptr(), plan.buf.numel() * 4,
                                        _stream(stream)))
    return plan


def _lora_args(X, A, B, plan, scale):
    """What both directions share; returns X's pitch, the device index and N, K, R, L."""
    torch = _tm()
    ldx = _first(X, "X", (torch.float16, torch.bfloat16))
    dev, dt = X.get_device(), X.dtype
    if not isinstance(plan, LoraPlan):
        raise TypeError("plan must be a LoraPlan (see lora_plan)")
    L = plan.L
    if A is None or B is None or A.dim() != 3 or B.dim() != 3:
        raise ValueError("A must be [L, R, K] and B [L, N, R]")
    R, N = A.shape[1], B.shape[1]
    M, K = X.shape
    if M != plan.M:
        raise ValueError(f"X has {M} rows, the plan is for {plan.M}")
    _like(A, "A", dt, (L, R, K), dev)
    _like(B, "B", dt, (L, N, R), dev)
    if plan.buf.get_device() != dev:
        raise ValueError(f"plan is on {plan.buf.device}, X on {X.device}")
    if scale is not None:
        _like(scale, "scale", torch.float32, (L,), dev)
    return ldx, dev, N, K, R, L


def lora_f16(X, A, B, plan: LoraPlan, scale=None, base=None, Y=None, V=None, stream=None):
    """Adapters' contribution added to a shared layer's output: with l the adapter of row m,
    V[m] = X[m] . A[l]^T and Y[m] = base[m] + scale[l] * V[m] . B[l]^T, fp16 or bf16.
    X [M, K], A [L, R, K], B [L, N, R], scale fp32 [L] (1 without), base [M, N] (0 without;
    Y may be base itself).  Returns (Y, V); V [M, R] is what lora_f16_bwd needs."""
    ldx, dev, N, K, R, L = _lora_args(X, A, B, plan, scale)
    dt, M = X.dtype, plan.M
    ldbase = 0 if base is None else _like(base, "base", dt, (M, N), dev)
    given = not (Y is None and V is None)
    if V is None:
        V = _new((M, R), dt, X, stream)
        ldv = V.stride(0)
    else:
        ldv = _like(V, "V", dt, (M, R), dev)
    if Y is None:
        Y = _new((M, N), dt, X if base is None else base, stream, pad=True)
        ldy = Y.stride(0)
    else:
        ldy = _like(Y, "Y", dt, (M, N), dev)
    if given:
        _apart(Y=Y, V=V)
    _check("lora_f16", lib().lora_f16(
        X.data_ptr(), ldx, A.data_ptr(), B.data_ptr(), _ptr(scale), plan.buf.data_ptr(), V.data_ptr(), ldv, _ptr(base),
        ldbase, Y.data_ptr(), ldy, M, N, K, R, L, _FLOAT_CODES[dt], _stream(stream)))
    return Y, V


def lora_f16_bwd(dY, X, V, A, B, plan: LoraPlan, scale=None, dbase=None, dX=None, dA=None, dB=None, workspace=None,
                 need_dx=True, stream=None):
    """Gradients of lora_f16: with U[m] = scale[l] * dY[m] . B[l], dX[m] = dbase[m] + U[m] . A[l]
    (dbase [M, K]: the shared layer's gradient of X, 0 without; dX may be dbase itself),
    dA[l] the sum of U[m]^T X[m] and dB[l] of scale[l] * dY[m]^T V[m] over l's rows.
    Returns (dX, dA, dB); dX is None with ``need_dx=False``."""
    ldx, dev, N, K, R, L = _lora_args(X, A, B, plan, scale)
    dt, M = X.dtype, plan.M
    lddy = _like(dY, "dY", dt, (M, N), dev)
    ldv = _like(V, "V", dt, (M, R), dev)
    lddb = 0 if dbase is None else _like(dbase, "dbase", dt, (M, K), dev)
    given = not (dX is None and dA is None and dB is None and workspace is None)
    if not need_dx and (dX is not None or dbase is not None):
        raise ValueError("need_dx=False takes neither dX nor dbase")
    lddx = 0
    if need_dx:
        if dX is None:
            dX = _new((M, K), dt, X, stream)
            lddx = dX.stride(0)
        else:
            lddx = _like(dX, "dX", dt, (M, K), dev)
    if dA is None:
        dA = _new((L, R, K), dt, A, stream)
    if dB is None:
        dB = _new((L, N, R), dt, B, stream)
    need = lib().lora_bwd_workspace_size(M, N, K, R, L)
    if workspace is None:
        workspace = _new((need,), _torch.uint8, X, stream)
    if given:
        _like(dA, "dA", dt, (L, R, K), dev)
        _like(dB, "dB", dt, (L, N, R), dev)
        _workspace(workspace, need, X.device)
        _apart(dX=dX, dA=dA, dB=dB, workspace=workspace)
    _check("lora_f16_bwd", lib().lora_f16_bwd(
        dY.data_ptr(), lddy, X.data_ptr(), ldx, V.data_ptr(), ldv, A.data_ptr(), B.data_ptr(), _ptr(scale),
        plan.buf.data_ptr(), _ptr(dbase), lddb, _ptr(dX), lddx, dA.data_ptr(), dB.data_ptr(), workspace.data_ptr(),
        _nbytes(workspace), M, N, K, R, L, _FLOAT_CODES[dt], _stream(stream)))
    return dX, dA, dB
