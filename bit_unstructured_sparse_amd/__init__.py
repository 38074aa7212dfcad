"""Bitmap-tiled int4 / fp16 sparse x dense matmul on AMD MI355X (gfx950).

A thin binding over ``libbitmap_spmm.so`` (C ABI in
``include/bitmap_spmm.h``): ctypes, and natively the steps that every call repeats
where ``_binding.so`` has been built. Host arrays are numpy; device memory and streams
come from PyTorch tensors. Every step of the SpMM runs in the library's HIP
kernels; there is no CPU fallback: if the library is missing, importing the
SpMM functions raises.

    import bit_unstructured_sparse_amd as bsp
    enc = bsp.encode(W_int8)                 # host, UnionSparse Sec. V-A with Q = 1
    dev = enc.to_device("cuda")              # torch tensors
    Xp  = bsp.pack_int4(X_int8)              # [N][ceil(K/2)] bytes
    Y   = bsp.spmm_w4a4(dev, torch.from_numpy(Xp).cuda(), N)   # int32 [N][M]
"""
from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass
from typing import NamedTuple, Optional

import numpy as np

__all__ = ["load_library", "encode", "pack_int4", "Encoded", "DeviceMatrix", "spmm_w4a4", "spmm_f16",
           "select", "describe", "workspace_bytes", "BspError", "ALGO_AUTO", "ALGO_ROWWAVE", "ALGO_MFMA",
           "ALGO_SPLITK",
           "INT4", "FP16", "INT8", "PAYLOAD_ALIGN", "MAX_N", "library_path", "KVCache", "new_kv_cache", "kv_append",
           "kv_gather", "attention_tree", "attention_workspace_bytes", "new_attention_workspace", "LoraAdapters",
           "spmm_f16_lora", "spmm_w4a4_dq_lora", "lora_workspace_bytes", "new_lora_workspace", "KVPages", "new_kv_pages",
           "KVStep", "kv_step", "rope_frequencies", "qk_norm_rope", "qk_norm_rope_append", "Tokens", "quantize_tokens",
           "dequantize_tokens", "EncodedInt8", "DenseInt8", "encode_int8", "gemm_workspace_bytes",
           "new_gemm_workspace", "describe_gemm", "gemm_w8a8"]

HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(HERE, "libbitmap_spmm.so")

OK, E_ARG, E_RANGE, E_CAPACITY, E_OVERFLOW, E_HIP, E_UNSUPPORTED = 0, 1, 2, 3, 4, 5, 6
INT4, FP16, INT2, INT8 = 0, 1, 2, 3      # INT8: caches, tokens and the dense product only
ALGO_AUTO, ALGO_ROWWAVE, ALGO_MFMA, ALGO_SPLITK = 0, 1, 2, 3
PAYLOAD_ALIGN = 16
MAX_N = 32

# Every symbol include/bitmap_spmm.h declares.
EXPORTS = ["encode_bitmap_tiles", "pack_int4_activations", "spmm_bitmap_w4a4", "spmm_bitmap_w4a4_algo",
           "spmm_bitmap_w4a4_ws", "spmm_bitmap_f16", "spmm_bitmap_f16_algo", "spmm_bitmap_f16_ws",
           "bsp_workspace_bytes", "bsp_select", "bsp_describe_selection", "bsp_describe_selection_ws", "bsp_describe_plan",
           "bsp_status_string", "bsp_version", "spmm_bitmap_f16_noalloc", "bsp_noalloc_scratch_bytes",
           "union_tile_count", "union_mask_words", "encode_union_tiles", "spmm_union_w4a4",
           "spmm_bitmap_w4a4_dq", "spmm_bitmap_w4a4_grouped", "spmm_bitmap_w2a4", "spmm_bitmap_w2a4_algo",
           "cbc_gtile_count", "encode_cbc_f16", "spmspv_cbc_workspace_bytes", "spmspv_cbc_f16",
           "kv_cache_append", "kv_cache_gather", "attention_tree_workspace_bytes", "attention_tree_f16",
           "lora_workspace_bytes", "spmm_bitmap_f16_lora", "spmm_bitmap_w4a4_dq_lora",
           "kv_pages_step", "qk_norm_rope_f16", "qk_norm_rope_append_f16", "quantize_tokens_f16",
           "dequantize_tokens_f16", "int8_tiles_bytes", "encode_int8_tiles", "gemm_w8a8_workspace_bytes",
           "gemm_w8a8_describe", "gemm_w8a8_dq"]


class BspError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


_lib = None


def load_library():
    """Load libbitmap_spmm.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(library_path):
            raise ImportError(f"{library_path} is missing; build it with "
                              "`python -m bit_unstructured_sparse_amd.build`")
        L = ctypes.CDLL(library_path)
        P, I64, I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        L.encode_bitmap_tiles.argtypes = [I32, P, I64, I64, I64, P, P, P, I64, P, P]
        L.encode_bitmap_tiles.restype = I32
        L.pack_int4_activations.argtypes, L.pack_int4_activations.restype = [P, I64, I64, I64, P], I32
        L.spmm_bitmap_w4a4.argtypes = [P, P, P, I64, I64, I64, P, I64, P, P]
        L.spmm_bitmap_w4a4.restype = I32
        L.spmm_bitmap_w4a4_algo.argtypes = [P, P, P, I64, I64, I64, P, I64, P, I32, P]
        L.spmm_bitmap_w4a4_algo.restype = I32
        L.spmm_bitmap_f16.argtypes = [P, P, P, I64, I64, I64, P, I64, P, P]
        L.spmm_bitmap_f16.restype = I32
        L.spmm_bitmap_f16_algo.argtypes = [P, P, P, I64, I64, I64, P, I64, P, I32, P]
        L.spmm_bitmap_f16_algo.restype = I32
        L.spmm_bitmap_w4a4_ws.argtypes = [P, P, P, I64, I64, I64, P, I64, P, P, I64, I32, P]
        L.spmm_bitmap_w4a4_ws.restype = I32
        L.spmm_bitmap_f16_ws.argtypes = [P, P, P, I64, I64, I64, P, I64, P, P, I64, I32, P]
        L.spmm_bitmap_f16_ws.restype = I32
        L.bsp_workspace_bytes.argtypes, L.bsp_workspace_bytes.restype = [I32, I64, I64, I64, I64, P], I32
        L.spmm_bitmap_f16_noalloc.argtypes = [P, P, P, I64, I64, I64, P, I64, P, I32, P]
        L.spmm_bitmap_f16_noalloc.restype = I32
        L.bsp_noalloc_scratch_bytes.argtypes, L.bsp_noalloc_scratch_bytes.restype = [], I64
        L.bsp_describe_selection_ws.argtypes = [I32, I64, I64, I64, I64, ctypes.c_char_p, ctypes.c_size_t]
        L.bsp_describe_selection_ws.restype = I32
        L.bsp_describe_plan.argtypes = [I32, I64, I64, I64, I64, I32, I32, ctypes.c_char_p, ctypes.c_size_t]
        L.bsp_describe_plan.restype = I32
        L.bsp_select.argtypes, L.bsp_select.restype = [I32, I64, I64, I64, I64], I32
        L.bsp_describe_selection.argtypes = [I32, I64, I64, I64, I64, ctypes.c_char_p, ctypes.c_size_t]
        L.bsp_describe_selection.restype = I32
        L.bsp_status_string.argtypes, L.bsp_status_string.restype = [I32], ctypes.c_char_p
        L.bsp_version.argtypes, L.bsp_version.restype = [], ctypes.c_char_p
        L.union_tile_count.argtypes, L.union_tile_count.restype = [I64, I64], I64
        L.union_mask_words.argtypes, L.union_mask_words.restype = [I32, I32], I32
        L.encode_union_tiles.argtypes = [P, I64, I64, I64, I32, I32, I32, P, P, P, P, I64, P, P]
        L.encode_union_tiles.restype = I32
        L.spmm_union_w4a4.argtypes = [P, P, P, P, I64, I32, I32, I64, I64, P, I64, P, P]
        L.spmm_union_w4a4.restype = I32
        L.spmm_bitmap_w4a4_dq.argtypes = [P, P, P, I64, I64, I64, P, I64, P, P, P, P]
        L.spmm_bitmap_w4a4_dq.restype = I32
        L.spmm_bitmap_w4a4_grouped.argtypes = [P, I32, I64, P]
        L.spmm_bitmap_w4a4_grouped.restype = I32
        L.spmm_bitmap_w2a4.argtypes = [P, P, P, I64, I64, I64, P, I64, P, P]
        L.spmm_bitmap_w2a4.restype = I32
        L.spmm_bitmap_w2a4_algo.argtypes = [P, P, P, I64, I64, I64, P, I64, P, I32, P]
        L.spmm_bitmap_w2a4_algo.restype = I32
        L.cbc_gtile_count.argtypes, L.cbc_gtile_count.restype = [I64, I64], I64
        L.encode_cbc_f16.argtypes = [P, I64, I64, I64, P, P, P, P, I64, P]
        L.encode_cbc_f16.restype = I32
        L.spmspv_cbc_workspace_bytes.argtypes, L.spmspv_cbc_workspace_bytes.restype = [I64, I64, I64, P], I32
        L.spmspv_cbc_f16.argtypes = [P, P, P, P, I64, I64, I64, P, I64, ctypes.c_float, P, P, I64, P]
        L.spmspv_cbc_f16.restype = I32
        F32 = ctypes.c_float
        L.kv_cache_append.argtypes, L.kv_cache_append.restype = [P, P, I64, P, I64, P, I64, P], I32
        L.kv_cache_gather.argtypes, L.kv_cache_gather.restype = [P, P, I64, P, I64, P, I64, P], I32
        L.attention_tree_workspace_bytes.argtypes = [P, I64, I64, I64, I64, P]
        L.attention_tree_workspace_bytes.restype = I32
        L.attention_tree_f16.argtypes = [P, I64, P, P, I64, P, P, I64, I64, I64, I64, P, F32, P, I64, P, I64, P]
        L.attention_tree_f16.restype = I32
        L.lora_workspace_bytes.argtypes, L.lora_workspace_bytes.restype = [I32, I64, I64, I64, I64, I64, P], I32
        L.spmm_bitmap_f16_lora.argtypes = [P, P, P, I64, I64, I64, P, I64, P, P, P, I64, P]
        L.spmm_bitmap_f16_lora.restype = I32
        L.spmm_bitmap_w4a4_dq_lora.argtypes = [P, P, P, I64, I64, I64, P, P, I64, P, P, P, P, P, I64, P]
        L.spmm_bitmap_w4a4_dq_lora.restype = I32
        L.kv_pages_step.argtypes, L.kv_pages_step.restype = [P, P, P, P, I64, P, P, P, P, P, P], I32
        L.qk_norm_rope_f16.argtypes = [P, I64, P, I64, I64, I64, I64, I64, P, P, I64, P, I64, P]
        L.qk_norm_rope_f16.restype = I32
        L.qk_norm_rope_append_f16.argtypes = [P, I64, P, I64, P, I64, I64, I64, P, P, P, P, I64, P]
        L.qk_norm_rope_append_f16.restype = I32
        L.quantize_tokens_f16.argtypes, L.quantize_tokens_f16.restype = [P, I32, P, I64, P], I32
        L.dequantize_tokens_f16.argtypes, L.dequantize_tokens_f16.restype = [P, I64, I32, P, I64, I64, P, I64, P], I32
        L.int8_tiles_bytes.argtypes, L.int8_tiles_bytes.restype = [I64, I64], I64
        L.encode_int8_tiles.argtypes, L.encode_int8_tiles.restype = [P, I64, I64, I64, P], I32
        L.gemm_w8a8_workspace_bytes.argtypes, L.gemm_w8a8_workspace_bytes.restype = [I64, I64, I64, P], I32
        L.gemm_w8a8_describe.argtypes = [I64, I64, I64, I32, ctypes.c_char_p, ctypes.c_size_t]
        L.gemm_w8a8_describe.restype = I32
        L.gemm_w8a8_dq.argtypes = [P, I64, I64, P, I64, I64, P, P, P, I64, P, I64, P]
        L.gemm_w8a8_dq.restype = I32
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return load_library().bsp_status_string(status).decode()


def _np_ptr(a: Optional[np.ndarray]):
    return None if a is None else a.ctypes.data_as(ctypes.c_void_p)


def _check(rc: int, what: str):
    if rc != OK:
        raise BspError(rc, what)


@dataclass
class Encoded:
    """Host-side BT64 stream: bitmaps uint64[M*T], offsets uint32[M*T+1],
    payload uint8[ceil(nnz/2)] (int4) or uint16[nnz] (fp16)."""
    dtype: int
    M: int
    K: int
    nnz: int
    bitmaps: np.ndarray
    offsets: np.ndarray
    payload: np.ndarray

    @property
    def T(self) -> int:
        return (self.K + 63) // 64

    @property
    def payload_bytes(self) -> int:
        return int(self.payload.nbytes)

    def to_device(self, device="cuda") -> "DeviceMatrix":
        import torch
        pad = (-self.payload_bytes) % PAYLOAD_ALIGN
        raw = np.zeros(self.payload_bytes + pad, np.uint8)
        raw[: self.payload_bytes] = self.payload.view(np.uint8)
        if raw.size == 0:
            raw = np.zeros(PAYLOAD_ALIGN, np.uint8)
        return DeviceMatrix(
            dtype=self.dtype, M=self.M, K=self.K, nnz=self.nnz,
            bitmaps=torch.from_numpy(self.bitmaps.view(np.int64)).to(device),
            offsets=torch.from_numpy(self.offsets.view(np.int32)).to(device),
            payload=torch.from_numpy(raw).to(device))


@dataclass
class DeviceMatrix:
    """The BT64 stream in device memory (torch tensors). ``payload`` is padded
    with zeros to a whole number of PAYLOAD_ALIGN bytes."""
    dtype: int
    M: int
    K: int
    nnz: int
    bitmaps: "object"
    offsets: "object"
    payload: "object"

    @property
    def T(self) -> int:
        return (self.K + 63) // 64

    def stream_bytes(self, with_offsets: bool = True) -> int:
        """Bytes of the encoded stream proper (unpadded payload)."""
        G = self.M * self.T
        pb = {INT4: (self.nnz + 1) // 2, INT2: (self.nnz + 3) // 4}.get(self.dtype, 2 * self.nnz)
        return 8 * G + (4 * (G + 1) if with_offsets else 0) + pb


def encode(W: np.ndarray, dtype: Optional[int] = None) -> Encoded:
    """Encode a dense host matrix: int8 (int4 values in [-8, 7]; with
    dtype=INT2, 2-bit values in [-2, 1]) or float16."""
    L = load_library()
    if W.dtype == np.int8:
        dt = INT2 if dtype == INT2 else INT4
    elif W.dtype == np.float16:
        dt = FP16
        W = W.view(np.uint16)
    elif W.dtype == np.uint16:
        dt = FP16
    else:
        raise TypeError("W must be int8 (int4 values) or float16")
    if W.ndim != 2:
        raise ValueError("W must be 2-D")
    M, K = W.shape
    ldw = W.strides[0] // W.itemsize if W.strides[1] == W.itemsize else None
    if ldw is None or ldw < K:
        W = np.ascontiguousarray(W)
        ldw = K
    nnz, nbytes = ctypes.c_int64(0), ctypes.c_int64(0)
    _check(L.encode_bitmap_tiles(dt, _np_ptr(W), M, K, ldw, None, None, None, 0,
                                 ctypes.byref(nnz), ctypes.byref(nbytes)), "encode_bitmap_tiles (size)")
    T = (K + 63) // 64
    bitmaps = np.empty(M * T, np.uint64)
    offsets = np.empty(M * T + 1, np.uint32)
    payload = np.empty(nnz.value if dt == FP16 else nbytes.value, np.uint16 if dt == FP16 else np.uint8)
    _check(L.encode_bitmap_tiles(dt, _np_ptr(W), M, K, ldw, _np_ptr(bitmaps), _np_ptr(offsets),
                                 _np_ptr(payload), payload.nbytes, ctypes.byref(nnz), ctypes.byref(nbytes)),
           "encode_bitmap_tiles")
    return Encoded(dt, M, K, int(nnz.value), bitmaps, offsets, payload)


def spmm_w2a4(W: DeviceMatrix, X, N: int, Y=None, algo: int = ALGO_AUTO, stream=None):
    """Y[n][m] = sum_k W[m][k] X[k][n] (int32) with 2-bit weights (a stream
    encoded with dtype=INT2). X: uint8 [N][ceil(K/2)] packed int4."""
    import torch
    if W.dtype != INT2:
        raise TypeError("spmm_w2a4 needs an INT2 DeviceMatrix")
    _check_dev(X, "X", torch.uint8, N * ((W.K + 1) // 2))
    if Y is None:
        Y = torch.empty((N, W.M), dtype=torch.int32, device=X.device)
    _check_dev(Y, "Y", torch.int32, N * W.M)
    rc = load_library().spmm_bitmap_w2a4_algo(
        _dptr(W.bitmaps), _dptr(W.offsets), _dptr(W.payload), W.payload.numel(), W.M, W.K,
        _dptr(X), N, _dptr(Y), algo, _stream_handle(stream))
    _check(rc, "spmm_bitmap_w2a4")
    return Y


def pack_int4(X: np.ndarray) -> np.ndarray:
    """int8 [N][K] activations in [-8, 7] -> packed uint8 [N][ceil(K/2)]."""
    if X.dtype != np.int8 or X.ndim != 2:
        raise TypeError("X must be a 2-D int8 array")
    X = np.ascontiguousarray(X)
    N, K = X.shape
    out = np.zeros((N, (K + 1) // 2), np.uint8)
    _check(load_library().pack_int4_activations(_np_ptr(X), N, K, K, _np_ptr(out)), "pack_int4_activations")
    return out


def _dptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream_handle(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check_dev(t, name, dtype, numel=None):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} elements, expected {numel}")


def _ws_args(workspace, index=None):
    if workspace is None:
        return None, 0
    import torch
    if not isinstance(workspace, torch.Tensor) or not workspace.is_cuda or not workspace.is_contiguous():
        raise TypeError("workspace must be a contiguous CUDA (HIP) tensor")
    if index is not None and workspace.get_device() != index:
        raise ValueError(f"workspace must be on device {index}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def spmm_w4a4(W: DeviceMatrix, X, N: int, Y=None, algo: int = ALGO_AUTO, stream=None, workspace=None):
    """Y[n][m] = sum_k W[m][k] X[k][n] (int32) on the GPU. X: uint8 [N][ceil(K/2)].
    workspace: an optional zero-initialised device tensor of at least
    workspace_bytes(...) bytes, 256-byte aligned (enables the split plans)."""
    import torch
    if W.dtype != INT4:
        raise TypeError("spmm_w4a4 needs an int4 DeviceMatrix")
    _check_dev(X, "X", torch.uint8, N * ((W.K + 1) // 2))
    if Y is None:
        Y = torch.empty((N, W.M), dtype=torch.int32, device=X.device)
    _check_dev(Y, "Y", torch.int32, N * W.M)
    wp, wb = _ws_args(workspace)
    rc = load_library().spmm_bitmap_w4a4_ws(
        _dptr(W.bitmaps), _dptr(W.offsets), _dptr(W.payload), W.payload.numel(), W.M, W.K,
        _dptr(X), N, _dptr(Y), wp, wb, algo, _stream_handle(stream))
    _check(rc, "spmm_bitmap_w4a4")
    return Y


def spmm_f16(W: DeviceMatrix, X, Y=None, algo: int = ALGO_AUTO, stream=None, workspace=None):
    """fp16 Y [N][M] = W X with fp32 accumulation. X: float16 [N][K]."""
    import torch
    if W.dtype != FP16:
        raise TypeError("spmm_f16 needs an fp16 DeviceMatrix")
    if X.dim() != 2 or X.shape[1] != W.K:
        raise ValueError("X must be [N][K]")
    N = int(X.shape[0])
    _check_dev(X, "X", torch.float16)
    if Y is None:
        Y = torch.empty((N, W.M), dtype=torch.float16, device=X.device)
    _check_dev(Y, "Y", torch.float16, N * W.M)
    wp, wb = _ws_args(workspace)
    rc = load_library().spmm_bitmap_f16_ws(
        _dptr(W.bitmaps), _dptr(W.offsets), _dptr(W.payload), W.payload.numel(), W.M, W.K,
        _dptr(X), N, _dptr(Y), wp, wb, algo, _stream_handle(stream))
    _check(rc, "spmm_bitmap_f16")
    return Y


# ---- dequant epilogue and grouped launch ----

GROUP_MAX = 8


class W4A4Item(ctypes.Structure):
    """bsp_w4a4_item of include/bitmap_spmm.h."""
    _fields_ = [("bitmaps", ctypes.c_void_p), ("offsets", ctypes.c_void_p), ("payload", ctypes.c_void_p),
                ("payload_bytes", ctypes.c_int64), ("M", ctypes.c_int64), ("X", ctypes.c_void_p),
                ("N", ctypes.c_int64), ("Y", ctypes.c_void_p), ("Yh", ctypes.c_void_p),
                ("scale_w", ctypes.c_void_p), ("scale_x", ctypes.c_void_p)]


def spmm_bitmap_w4a4_dq(W: DeviceMatrix, X, N: int, scale_w, scale_x, Yh=None, stream=None):
    """fp16 Yh [N][M] = fp16(fp32(fp32(W X) * scale_w[m]) * scale_x[n]), the
    dequant step fused into the int4 SpMM. scale_w: float32 [M], scale_x:
    float32 [N] (device)."""
    import torch
    if W.dtype != INT4:
        raise TypeError("spmm_bitmap_w4a4_dq needs an int4 DeviceMatrix")
    _check_dev(X, "X", torch.uint8, N * ((W.K + 1) // 2))
    _check_dev(scale_w, "scale_w", torch.float32, W.M)
    _check_dev(scale_x, "scale_x", torch.float32, N)
    if Yh is None:
        Yh = torch.empty((N, W.M), dtype=torch.float16, device=X.device)
    _check_dev(Yh, "Yh", torch.float16, N * W.M)
    rc = load_library().spmm_bitmap_w4a4_dq(
        _dptr(W.bitmaps), _dptr(W.offsets), _dptr(W.payload), W.payload.numel(), W.M, W.K, _dptr(X), N,
        _dptr(scale_w), _dptr(scale_x), _dptr(Yh), _stream_handle(stream))
    _check(rc, "spmm_bitmap_w4a4_dq")
    return Yh


def spmm_bitmap_w4a4_grouped(items, stream=None):
    """One launch for several int4 matrices of one K. items: a list of dicts
    with W (DeviceMatrix), X (uint8 [N][ceil(K/2)]), N, and either Y (int32
    [N][M]) or Yh (fp16 [N][M]) with scale_w (float32 [M]) and scale_x
    (float32 [N]). Returns the list of outputs."""
    import torch
    if not items:
        raise ValueError("no items")
    K = items[0]["W"].K
    arr = (W4A4Item * len(items))()
    outs = []
    for i, it in enumerate(items):
        W, X, N = it["W"], it["X"], int(it["N"])
        if W.K != K or W.dtype != INT4:
            raise ValueError("grouped items must be int4 matrices of one K")
        _check_dev(X, "X", torch.uint8, N * ((K + 1) // 2))
        Y, Yh = it.get("Y"), it.get("Yh")
        sw, sx = it.get("scale_w"), it.get("scale_x")
        if sw is not None:
            _check_dev(sw, "scale_w", torch.float32, W.M)
            _check_dev(sx, "scale_x", torch.float32, N)
            if Yh is None:
                Yh = torch.empty((N, W.M), dtype=torch.float16, device=X.device)
            _check_dev(Yh, "Yh", torch.float16, N * W.M)
            outs.append(Yh)
        else:
            if Y is None:
                Y = torch.empty((N, W.M), dtype=torch.int32, device=X.device)
            _check_dev(Y, "Y", torch.int32, N * W.M)
            outs.append(Y)
        arr[i] = W4A4Item(_dptr(W.bitmaps), _dptr(W.offsets), _dptr(W.payload), W.payload.numel(), W.M, _dptr(X), N,
                          _dptr(Y) if sw is None else None, _dptr(Yh) if sw is not None else None, _dptr(sw),
                          _dptr(sx))
    rc = load_library().spmm_bitmap_w4a4_grouped(ctypes.cast(arr, ctypes.c_void_p), len(items), K,
                                                 _stream_handle(stream))
    _check(rc, "spmm_bitmap_w4a4_grouped")
    return outs


# ---- Tiled-CBC format with dynamic activation pruning (fp16) ----

CBC_TILE = (256, 64)
CBC_MAX_N = 8


@dataclass
class CbcEncoded:
    """Host-side Tiled-CBC stream: tile_offsets uint32[n_gt + 1], colinfo
    uint32[n_gt * 64], bitmaps uint64[n_gt * 256], values fp16 bits [nnz]."""
    M: int
    K: int
    nnz: int
    tile_offsets: np.ndarray
    colinfo: np.ndarray
    bitmaps: np.ndarray
    values: np.ndarray

    def storage_bytes(self) -> int:
        return int(self.tile_offsets.nbytes + self.colinfo.nbytes + self.bitmaps.nbytes + self.values.nbytes)

    def to_device(self, device="cuda") -> "CbcDevice":
        import torch
        vb = self.values.nbytes
        raw = np.zeros(max(PAYLOAD_ALIGN, vb + (-vb) % PAYLOAD_ALIGN), np.uint8)
        raw[:vb] = self.values.view(np.uint8)
        return CbcDevice(self.M, self.K, self.nnz,
                         torch.from_numpy(self.tile_offsets.view(np.int32)).to(device),
                         torch.from_numpy(self.colinfo.view(np.int32)).to(device),
                         torch.from_numpy(self.bitmaps.view(np.int64)).to(device),
                         torch.from_numpy(raw).to(device))


@dataclass
class CbcDevice:
    M: int
    K: int
    nnz: int
    tile_offsets: "object"
    colinfo: "object"
    bitmaps: "object"
    values: "object"       # uint8, padded to PAYLOAD_ALIGN


def cbc_gtile_count(M: int, K: int) -> int:
    return int(load_library().cbc_gtile_count(M, K))


def encode_cbc_f16(W: np.ndarray) -> CbcEncoded:
    L = load_library()
    W = np.ascontiguousarray(W)
    if W.dtype == np.float16:
        W = W.view(np.uint16)
    if W.dtype != np.uint16 or W.ndim != 2:
        raise TypeError("W must be a 2-D float16 (or uint16 bits) array")
    M, K = W.shape
    nnz = ctypes.c_int64(0)
    _check(L.encode_cbc_f16(_np_ptr(W), M, K, K, None, None, None, None, 0, ctypes.byref(nnz)), "encode_cbc_f16 (size)")
    ngt = cbc_gtile_count(M, K)
    to = np.zeros(ngt + 1, np.uint32)
    ci = np.zeros(ngt * 64, np.uint32)
    bm = np.zeros(ngt * 256, np.uint64)
    vals = np.zeros(nnz.value, np.uint16)
    _check(L.encode_cbc_f16(_np_ptr(W), M, K, K, _np_ptr(to), _np_ptr(ci), _np_ptr(bm), _np_ptr(vals), vals.size,
                            ctypes.byref(nnz)), "encode_cbc_f16")
    return CbcEncoded(M, K, int(nnz.value), to, ci, bm, vals)


def spmspv_cbc_workspace_bytes(M: int, K: int, N: int) -> int:
    b = ctypes.c_int64(0)
    _check(load_library().spmspv_cbc_workspace_bytes(M, K, N, ctypes.byref(b)), "spmspv_cbc_workspace_bytes")
    return int(b.value)


def new_cbc_workspace(M: int, K: int, N: int, device="cuda"):
    import torch
    n = spmspv_cbc_workspace_bytes(M, K, N)
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=device) if n else None


def spmspv_cbc_f16(D: CbcDevice, X, threshold: float, Y=None, workspace=None, stream=None):
    """fp16 Y [N][M] = W X' with X' = X where |x| > threshold, else 0 (dynamic
    activation pruning; the all-pruned columns of W are not read)."""
    import torch
    if X.dim() != 2 or X.shape[1] != D.K:
        raise ValueError("X must be [N][K]")
    N = int(X.shape[0])
    _check_dev(X, "X", torch.float16)
    if Y is None:
        Y = torch.empty((N, D.M), dtype=torch.float16, device=X.device)
    _check_dev(Y, "Y", torch.float16, N * D.M)
    wp, wb = _ws_args(workspace)
    rc = load_library().spmspv_cbc_f16(
        _dptr(D.tile_offsets), _dptr(D.colinfo), _dptr(D.bitmaps), _dptr(D.values), D.values.numel(), D.M, D.K,
        _dptr(X), N, ctypes.c_float(threshold), _dptr(Y), wp, wb, _stream_handle(stream))
    _check(rc, "spmspv_cbc_f16")
    return Y


# ---- union-mask (IE-BME) format: 16 x 64 local tiles, ra x ca areas ----

UNION_MAX_K = 32768


@dataclass
class UnionEncoded:
    """Host-side union-mask stream: ubitmaps uint64[nlt * words], offsets
    uint32[nlt + 1], rowpos uint64[nlt], payload uint8[ceil(nvals / 2)]."""
    M: int
    K: int
    ra: int
    ca: int
    nvals: int
    ubitmaps: np.ndarray
    offsets: np.ndarray
    rowpos: np.ndarray
    payload: np.ndarray

    @property
    def nlt(self) -> int:
        return int(self.rowpos.size)

    def stream_bytes(self) -> int:
        """Bytes of the encoded stream proper: mask words, offsets, rowpos, payload."""
        return int(self.ubitmaps.nbytes + self.offsets.nbytes + self.rowpos.nbytes + self.payload.nbytes)

    def to_device(self, device="cuda") -> "UnionDevice":
        import torch
        pb = self.payload.nbytes
        raw = np.zeros(max(PAYLOAD_ALIGN, pb + (-pb) % PAYLOAD_ALIGN), np.uint8)
        raw[:pb] = self.payload
        return UnionDevice(self.M, self.K, self.ra, self.ca, self.nvals,
                           torch.from_numpy(self.ubitmaps.view(np.int64)).to(device),
                           torch.from_numpy(self.offsets.view(np.int32)).to(device),
                           torch.from_numpy(self.rowpos.view(np.int64)).to(device),
                           torch.from_numpy(raw).to(device))


@dataclass
class UnionDevice:
    """The union-mask stream in device memory; payload padded with zeros to a
    whole number of PAYLOAD_ALIGN bytes."""
    M: int
    K: int
    ra: int
    ca: int
    nvals: int
    ubitmaps: "object"
    offsets: "object"
    rowpos: "object"
    payload: "object"


def union_tile_count(M: int, K: int) -> int:
    return int(load_library().union_tile_count(M, K))


def union_mask_words(ra: int, ca: int) -> int:
    return int(load_library().union_mask_words(ra, ca))


def encode_union_tiles(W: np.ndarray, ra: int = 2, ca: int = 2, reorder: bool = True) -> UnionEncoded:
    """Union-mask encoding of an int8 (int4 values) host matrix, with
    bitmap-aware row reordering of every local tile when ``reorder``."""
    L = load_library()
    if W.dtype != np.int8 or W.ndim != 2:
        raise TypeError("W must be a 2-D int8 array of int4 values")
    W = np.ascontiguousarray(W)
    M, K = W.shape
    nv, nb = ctypes.c_int64(0), ctypes.c_int64(0)
    _check(L.encode_union_tiles(_np_ptr(W), M, K, K, ra, ca, int(reorder), None, None, None, None, 0,
                                ctypes.byref(nv), ctypes.byref(nb)), "encode_union_tiles (size)")
    nlt, words = union_tile_count(M, K), union_mask_words(ra, ca)
    ub = np.zeros(nlt * words, np.uint64)
    off = np.zeros(nlt + 1, np.uint32)
    rp = np.zeros(nlt, np.uint64)
    pl = np.zeros(nb.value, np.uint8)
    _check(L.encode_union_tiles(_np_ptr(W), M, K, K, ra, ca, int(reorder), _np_ptr(ub), _np_ptr(off), _np_ptr(rp),
                                _np_ptr(pl), pl.nbytes, ctypes.byref(nv), ctypes.byref(nb)), "encode_union_tiles")
    return UnionEncoded(M, K, ra, ca, int(nv.value), ub, off, rp, pl)


def spmm_union_w4a4(U: UnionDevice, X, N: int, Y=None, stream=None):
    """Y[n][m] = sum_k W[m][k] X[k][n] (int32) with W in the union-mask
    format. X: uint8 [N][ceil(K/2)] packed int4."""
    import torch
    _check_dev(X, "X", torch.uint8, N * ((U.K + 1) // 2))
    if Y is None:
        Y = torch.empty((N, U.M), dtype=torch.int32, device=X.device)
    _check_dev(Y, "Y", torch.int32, N * U.M)
    rc = load_library().spmm_union_w4a4(
        _dptr(U.ubitmaps), _dptr(U.offsets), _dptr(U.rowpos), _dptr(U.payload), U.payload.numel(), U.ra, U.ca,
        U.M, U.K, _dptr(X), N, _dptr(Y), _stream_handle(stream))
    _check(rc, "spmm_union_w4a4")
    return Y


def select(dtype: int, M: int, K: int, N: int, nnz: int = -1) -> int:
    return int(load_library().bsp_select(dtype, M, K, N, nnz))


def describe(dtype: int, M: int, K: int, N: int, nnz: int = -1, workspace: bool = False,
             algo: int = ALGO_AUTO) -> str:
    """The plan (kernel and launch shape) of the plain entry points, or with
    workspace=True of the *_ws entry points given a workspace; for an
    explicit algo, the plan that choice takes (BspError if it cannot run)."""
    buf = ctypes.create_string_buffer(384)
    if algo != ALGO_AUTO:
        _check(load_library().bsp_describe_plan(dtype, M, K, N, nnz, algo, int(workspace), buf, 384),
               "bsp_describe_plan")
        return buf.value.decode()
    fn = load_library().bsp_describe_selection_ws if workspace else load_library().bsp_describe_selection
    _check(fn(dtype, M, K, N, nnz, buf, 384), "bsp_describe_selection")
    return buf.value.decode()


def workspace_bytes(dtype: int, M: int, K: int, N: int, nnz: int = -1) -> int:
    """Bytes of workspace the *_ws entry points want for a problem (0: none)."""
    out = ctypes.c_int64(0)
    _check(load_library().bsp_workspace_bytes(dtype, M, K, N, nnz, ctypes.byref(out)), "bsp_workspace_bytes")
    return int(out.value)


def new_workspace(dtype: int, M: int, K: int, N: int, nnz: int = -1, device="cuda"):
    """A zero-filled device workspace for the split plans (None if none is needed)."""
    import torch
    n = workspace_bytes(dtype, M, K, N, nnz)
    if n == 0:
        return None
    return torch.zeros(n, dtype=torch.uint8, device=device)


# ---- paged key/value cache, quantised as it is written ----

TREE_MAX = 64
PAGES_MAX_SEQUENCES = 4096


class _KVCacheDesc(ctypes.Structure):
    """bsp_kv_cache of include/bitmap_spmm.h."""
    _fields_ = [("dtype", ctypes.c_int), ("num_pages", ctypes.c_int64), ("kv_heads", ctypes.c_int64),
                ("page_size", ctypes.c_int64), ("head_dim", ctypes.c_int64), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]


@dataclass(frozen=True)
class KVCache:
    """Paged cache tensors (their contents change, the tensors do not): k, v [pages][kv_heads][page_size][row] (float16
    [head_dim] for FP16, uint8 [head_dim] for INT8, uint8 [head_dim / 2] for
    INT4) and, for the quantised kinds, k_scale, v_scale int32
    [pages][kv_heads][page_size] (step as bfloat16 in the high half, offset as
    float16 in the low half)."""
    dtype: int
    k: "object"
    v: "object"
    k_scale: "object" = None
    v_scale: "object" = None

    def __post_init__(self):
        import torch
        if self.dtype not in (FP16, INT8, INT4):
            raise ValueError("a cache is FP16, INT8 or INT4")
        if self.k.dim() != 4 or self.v.shape != self.k.shape:
            raise ValueError("k and v must be [pages][kv_heads][page_size][row] of one shape")
        for n in ("k", "v"):
            _check_dev(getattr(self, n), n, torch.float16 if self.dtype == FP16 else torch.uint8)
        for n in ("k_scale", "v_scale"):
            w = getattr(self, n)
            if self.dtype == FP16:
                if w is not None:
                    raise ValueError("an FP16 cache has no scale words")
            else:
                _check_dev(w, n, torch.int32)
                if w.shape != self.k.shape[:3]:
                    raise ValueError(f"{n} must be [pages][kv_heads][page_size]")
        if len({t.device for t in (self.k, self.v, self.k_scale, self.v_scale) if t is not None}) != 1:
            raise ValueError("the cache's tensors must lie on one device")
        pages, heads, page_size, row = (int(n) for n in self.k.shape)
        dim = 2 * row if self.dtype == INT4 else row
        desc = _KVCacheDesc(self.dtype, pages, heads, page_size, dim, _dptr(self.k), _dptr(self.v),
                            _dptr(self.k_scale), _dptr(self.v_scale))
        for name, value in (("num_pages", pages), ("kv_heads", heads), ("page_size", page_size), ("head_dim", dim),
                            ("device", self.k.device), ("_index", self.k.get_device()), ("_desc", desc),
                            ("_ref", ctypes.addressof(desc))):
            object.__setattr__(self, name, value)


def new_kv_cache(dtype: int, num_pages: int, kv_heads: int, page_size: int, head_dim: int, device="cuda") -> KVCache:
    """A cache of num_pages empty (zero) pages."""
    import torch
    if dtype not in (FP16, INT8, INT4):
        raise ValueError("a cache is FP16, INT8 or INT4")
    shape = (num_pages, kv_heads, page_size)
    row = head_dim // 2 if dtype == INT4 else head_dim

    def codes():
        return torch.zeros(shape + (row,), dtype=torch.float16 if dtype == FP16 else torch.uint8, device=device)

    def words():
        return None if dtype == FP16 else torch.zeros(shape, dtype=torch.int32, device=device)

    return KVCache(dtype, codes(), codes(), words(), words())


def _rows(t, name, n, heads, dim, index) -> int:
    """Check a float16 [n][heads][dim] tensor (n None: any) whose rows may be
    strided by token; returns the stride between tokens."""
    import torch
    width = heads * dim
    # the common case in few steps; _rows_error names what is wrong
    if isinstance(t, torch.Tensor) and t.dtype is torch.float16 and t.get_device() == index and t.dim() == 3:
        m, h, d = t.shape
        if h == heads and d == dim and (n is None or m == n):
            if t.is_contiguous():
                return width
            s0, s1, s2 = t.stride()
            if s2 == 1 and (heads == 1 or s1 == dim):
                if m <= 1:
                    return width
                if s0 >= width:
                    return s0
    raise _rows_error(t, name, n, heads, dim, index)


def _rows_error(t, name, n, heads, dim, index):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        return TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype != torch.float16:
        return TypeError(f"{name} must be torch.float16, got {t.dtype}")
    if t.get_device() != index:
        return ValueError(f"{name} must be on device {index}")
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != dim or (n is not None and t.shape[0] != n):
        return ValueError(f"{name} must be [{'tokens' if n is None else n}][{heads}][{dim}], got {tuple(t.shape)}")
    return ValueError(f"{name}: the heads of a token must be contiguous, and tokens must not overlap")


def _flat(t, name, dtype, numel, index) -> int:
    """Check a contiguous device tensor; returns its address."""
    import torch
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index and t.is_contiguous() and \
            t.numel() == numel:
        return t.data_ptr()
    _check_dev(t, name, dtype, numel)
    raise ValueError(f"{name} must be on device {index}")


def _launch(fn, index: int, stream, *args) -> int:
    """Calls an entry point on a stream, by default the device's current one (by
    its handle alone: the Stream object around it costs as much as a launch),
    with the tensors' device as the current one: kernels go to the current
    device, and its default stream has the same handle as every other device's."""
    import torch
    if not _native_tried:
        _use_native()
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(index)
    elif stream.device_index == index:
        handle = stream.cuda_stream
    else:
        raise ValueError(f"the stream must be one of device {index}")
    if torch._C._cuda_getDevice() == index:
        return fn(*args, handle)
    with torch.cuda.device(index):
        return fn(*args, handle)


_native_tried = False


def _use_native() -> None:
    """From the first launch on, the steps above and the outputs' allocation natively (_binding.so), where it has
    been built: the same results, and these functions for every case that is not the common one."""
    global _native_tried, _flat, _rows, _matrix_rows, _new_output, _launch
    if _native_tried:
        return
    _native_tried = True
    try:
        import torch
        from . import _binding
    except ImportError:
        return
    L = load_library()
    if not isinstance(L, ctypes.CDLL):
        return
    _binding.bind(L._handle, {name: getattr(L, name) for name in EXPORTS},
                  (_flat, _rows, _matrix_rows, _new_output, _launch), torch)
    _flat, _rows, _matrix_rows, _new_output, _launch = (_binding.flat, _binding.rows, _binding.matrix_rows,
                                                        _binding.new_output, _binding.launch)


def _weights_on(W: DeviceMatrix, index: int) -> None:
    if not W.bitmaps.get_device() == W.offsets.get_device() == W.payload.get_device() == index:
        raise ValueError(f"the projection must be on device {index}")


def _new_output(shape, dtype, device, stream):
    """A tensor for a call to write on `stream`. It is taken from that stream's
    memory: a block of the current stream's may still be in use by what was
    queued there. The current stream, where the caller will read it, is noted
    for the time it is freed."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _call_workspace(n: int, device, stream):
    """A zero-filled workspace for one call on `stream`: cleared on that stream,
    ahead of the call, and free for that stream's later work once dropped."""
    import torch
    if n == 0:
        return None
    if stream is None:
        return torch.zeros(n, dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.zeros(n, dtype=torch.uint8, device=device)


def kv_append(cache: KVCache, K, V, slots, stream=None) -> None:
    """Quantise the rows K, V (float16 [n][kv_heads][head_dim], a token's heads
    contiguous) into cache slots (int64 [n], page * page_size + offset; a slot
    outside the cache is skipped)."""
    import torch
    heads, dim, index = cache.kv_heads, cache.head_dim, cache._index
    ks = _rows(K, "K", None, heads, dim, index)
    n = K.shape[0]
    vs = _rows(V, "V", n, heads, dim, index)
    rc = _launch(load_library().kv_cache_append, index, stream, cache._ref, K.data_ptr(), ks, V.data_ptr(), vs,
                 _flat(slots, "slots", torch.int64, n, index), n)
    _check(rc, "kv_cache_append")


def kv_gather(cache: KVCache, slots, K=None, V=None, stream=None):
    """The rows of the slots (int64 [n]) as float16 K, V [n][kv_heads][head_dim]
    (zeros for a slot outside the cache)."""
    import torch
    heads, dim, index = cache.kv_heads, cache.head_dim, cache._index
    n = slots.numel()
    at = _flat(slots, "slots", torch.int64, n, index)
    if K is None:
        K = _new_output((n, heads, dim), torch.float16, cache.device, stream)
    if V is None:
        V = _new_output((n, heads, dim), torch.float16, cache.device, stream)
    ks, vs = _rows(K, "K", n, heads, dim, index), _rows(V, "V", n, heads, dim, index)
    rc = _launch(load_library().kv_cache_gather, index, stream, cache._ref, at, n, K.data_ptr(), ks, V.data_ptr(), vs)
    _check(rc, "kv_cache_gather")
    return K, V


# ---- attention of drafted token trees over the cache ----

def attention_workspace_bytes(cache: KVCache, B: int, max_q: int, q_heads: int, table_width: int) -> int:
    """Bytes of workspace attention_tree uses to split the cached tokens."""
    out = ctypes.c_int64(0)
    _check(load_library().attention_tree_workspace_bytes(cache._ref, table_width, B, max_q, q_heads,
                                                         ctypes.byref(out)), "attention_tree_workspace_bytes")
    return int(out.value)


def new_attention_workspace(cache: KVCache, B: int, max_q: int, q_heads: int, table_width: int, device="cuda"):
    """A zero-filled workspace for attention_tree (None if none is used).
    It is cleared on the current stream: calls on another one wait for that."""
    import torch
    n = attention_workspace_bytes(cache, B, max_q, q_heads, table_width)
    return torch.zeros(n, dtype=torch.uint8, device=device) if n else None


def attention_tree(Q, cache: KVCache, block_table, kv_lens, q_start, max_q: int, tree_mask=None, scale=None, O=None,
                   workspace=None, stream=None):
    """float16 O [rows][q_heads][head_dim]: attention of each sequence's drafted
    tokens over its cached tokens. Q: float16 [rows][q_heads][head_dim];
    block_table: int32 [B][width]; kv_lens: int32 [B], cached tokens, the drafted
    ones last; q_start: int32 [B + 1], the rows of sequence b are q_start[b] up to
    q_start[b + 1] (at most max_q <= TREE_MAX of them); tree_mask: int64 [rows],
    bit j of row i's word: drafted token j is seen (None: a chain); scale: default
    head_dim ** -0.5. workspace: new_attention_workspace(...), or None for no
    split over the cached tokens."""
    import torch
    dim, index = cache.head_dim, cache._index
    if Q.dim() != 3:
        raise ValueError("Q must be [rows][q_heads][head_dim]")
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B][width]")
    rows, hq, _ = Q.shape
    B, width = block_table.shape
    qs = _rows(Q, "Q", None, hq, dim, index)
    if O is None:
        O = _new_output((rows, hq, dim), torch.float16, cache.device, stream)
    os_ = _rows(O, "O", rows, hq, dim, index)
    wp, wb = _ws_args(workspace, index)
    i32 = torch.int32
    rc = _launch(
        load_library().attention_tree_f16, index, stream,
        Q.data_ptr(), qs, cache._ref, _flat(block_table, "block_table", i32, B * width, index), width,
        _flat(kv_lens, "kv_lens", i32, B, index), _flat(q_start, "q_start", i32, B + 1, index), B, rows, max_q, hq,
        None if tree_mask is None else _flat(tree_mask, "tree_mask", torch.int64, rows, index),
        dim ** -0.5 if scale is None else scale, O.data_ptr(), os_, wp, wb)
    _check(rc, "attention_tree_f16")
    return O


# ---- low-rank adapters beside a shared projection ----

class _LoraDesc(ctypes.Structure):
    """bsp_lora of include/bitmap_spmm.h."""
    _fields_ = [("adapters", ctypes.c_int64), ("rank", ctypes.c_int64), ("A", ctypes.c_void_p),
                ("B", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("ranks", ctypes.c_void_p),
                ("index", ctypes.c_void_p)]


@dataclass(frozen=True)
class LoraAdapters:
    """The adapters of one projection: A float16 [adapters][R][K], B float16
    [adapters][M][R] (R a multiple of 8, at most 256); scale float32 [adapters]
    (None: 1); rank int32 [adapters], the rows of A in use (None: R). A tensor
    given another storage is taken up, and checked, by the next call."""
    A: "object"
    B: "object"
    scale: "object" = None
    rank: "object" = None

    def __post_init__(self):
        import torch
        if self.A.dim() != 3 or self.B.dim() != 3 or self.A.shape[0] != self.B.shape[0] or \
                self.A.shape[1] != self.B.shape[2]:
            raise ValueError("A must be [adapters][R][K] and B [adapters][M][R]")
        _check_dev(self.A, "A", torch.float16)
        n, R, K = (int(x) for x in self.A.shape)
        index = self.A.get_device()
        _flat(self.B, "B", torch.float16, self.B.numel(), index)
        if self.scale is not None:
            _flat(self.scale, "scale", torch.float32, n, index)
        if self.rank is not None:
            _flat(self.rank, "rank", torch.int32, n, index)
        at = (_dptr(self.A), _dptr(self.B), _dptr(self.scale), _dptr(self.rank))
        for name, value in (("adapters", n), ("R", R), ("K", K), ("M", int(self.B.shape[1])), ("_index", index),
                            ("_at", at), ("_fixed", (n, R) + at)):
            object.__setattr__(self, name, value)

    def _desc(self, W, index, N) -> _LoraDesc:
        import torch
        scale, rank = self.scale, self.rank
        if (self.A.data_ptr(), self.B.data_ptr(), None if scale is None else scale.data_ptr(),
                None if rank is None else rank.data_ptr()) != self._at:
            self.__post_init__()
        if self.K != W.K or self.M != W.M:
            raise ValueError(f"the adapters are for a {self.M} x {self.K} projection, not {W.M} x {W.K}")
        return _LoraDesc(*self._fixed, _flat(index, "index", torch.int32, N, self._index))


def lora_workspace_bytes(dtype: int, M: int, K: int, N: int, rank: int, nnz: int = -1) -> int:
    """Bytes of workspace the adapter entry points need."""
    out = ctypes.c_int64(0)
    _check(load_library().lora_workspace_bytes(dtype, M, K, N, nnz, rank, ctypes.byref(out)), "lora_workspace_bytes")
    return int(out.value)


def _lora_bytes(W: DeviceMatrix, N: int, adapters: LoraAdapters) -> int:
    return lora_workspace_bytes(W.dtype, W.M, W.K, N, adapters.R, W.nnz)


def new_lora_workspace(W: DeviceMatrix, N: int, adapters: LoraAdapters, device="cuda"):
    """A zero-filled workspace for the adapter entry points (None if empty).
    It is cleared on the current stream: calls on another one wait for that."""
    import torch
    n = _lora_bytes(W, N, adapters)
    return torch.zeros(n, dtype=torch.uint8, device=device) if n else None


def spmm_f16_lora(W: DeviceMatrix, X, adapters: LoraAdapters, index, Y=None, workspace=None, stream=None):
    """fp16 Y [N][M] = W x_n + scale[a] B_a (A_a x_n), a = index[n] (int32 [N];
    negative: no adapter). X: float16 [N][K]. workspace: new_lora_workspace(...)
    (one is made for the call, on its stream, when not given)."""
    import torch
    if W.dtype != FP16:
        raise TypeError("spmm_f16_lora needs an fp16 DeviceMatrix")
    if X.dim() != 2 or X.shape[1] != W.K:
        raise ValueError("X must be [N][K]")
    N, dev = X.shape[0], adapters._index
    _weights_on(W, dev)
    x = _flat(X, "X", torch.float16, N * W.K, dev)
    d = adapters._desc(W, index, N)
    if Y is None:
        Y = _new_output((N, W.M), torch.float16, X.device, stream)
    y = _flat(Y, "Y", torch.float16, N * W.M, dev)
    if workspace is None:
        workspace = _call_workspace(_lora_bytes(W, N, adapters), X.device, stream)
    wp, wb = _ws_args(workspace, dev)
    rc = _launch(
        load_library().spmm_bitmap_f16_lora, dev, stream,
        W.bitmaps.data_ptr(), W.offsets.data_ptr(), W.payload.data_ptr(), W.payload.numel(), W.M, W.K, x, N,
        ctypes.byref(d), y, wp, wb)
    _check(rc, "spmm_bitmap_f16_lora")
    return Y


def spmm_w4a4_dq_lora(W: DeviceMatrix, X, X16, scale_w, scale_x, adapters: LoraAdapters, index, Yh=None,
                      workspace=None, stream=None):
    """fp16 Yh [N][M] = (W x_n) * scale_w[m] * scale_x[n] + scale[a] B_a (A_a
    x16_n): the dequantised int4 product of spmm_bitmap_w4a4_dq with adapters on
    the float16 activations. X: uint8 [N][ceil(K/2)] packed int4; X16: float16
    [N][K]."""
    import torch
    if W.dtype != INT4:
        raise TypeError("spmm_w4a4_dq_lora needs an int4 DeviceMatrix")
    if X16.dim() != 2 or X16.shape[1] != W.K:
        raise ValueError("X16 must be [N][K]")
    N, dev = X16.shape[0], adapters._index
    _weights_on(W, dev)
    x16 = _flat(X16, "X16", torch.float16, N * W.K, dev)
    x = _flat(X, "X", torch.uint8, N * ((W.K + 1) // 2), dev)
    sw, sx = _flat(scale_w, "scale_w", torch.float32, W.M, dev), _flat(scale_x, "scale_x", torch.float32, N, dev)
    d = adapters._desc(W, index, N)
    if Yh is None:
        Yh = _new_output((N, W.M), torch.float16, X16.device, stream)
    y = _flat(Yh, "Yh", torch.float16, N * W.M, dev)
    if workspace is None:
        workspace = _call_workspace(_lora_bytes(W, N, adapters), X16.device, stream)
    wp, wb = _ws_args(workspace, dev)
    rc = _launch(
        load_library().spmm_bitmap_w4a4_dq_lora, dev, stream,
        W.bitmaps.data_ptr(), W.offsets.data_ptr(), W.payload.data_ptr(), W.payload.numel(), W.M, W.K, x, x16, N, sw, sx,
        ctypes.byref(d), y, wp, wb)
    _check(rc, "spmm_bitmap_w4a4_dq_lora")
    return Yh


# ---- pages, slots and positions of a step, made on the GPU ----

class _KVPagesDesc(ctypes.Structure):
    """bsp_kv_pages of include/bitmap_spmm.h."""
    _fields_ = [("sequences", ctypes.c_int64), ("table_width", ctypes.c_int64), ("page_size", ctypes.c_int64),
                ("pool", ctypes.c_int64), ("block_table", ctypes.c_void_p), ("lens", ctypes.c_void_p),
                ("held", ctypes.c_void_p), ("free_pages", ctypes.c_void_p)]


@dataclass(frozen=True)
class KVPages:
    """Which pages of a cache each sequence holds, in device memory and updated there by kv_step: block_table int32
    [B][width] (as attention_tree takes it), lens int32 [B] tokens cached, held int32 [B] pages held, free int32
    [2 + pool]: the number of free pages, a counter of the call's own (0), the free pages (the next to be taken last).
    Calls on the same pages must be ordered on one stream."""
    block_table: "object"
    lens: "object"
    held: "object"
    free: "object"
    page_size: int

    def __post_init__(self):
        import torch
        if self.block_table.dim() != 2:
            raise ValueError("block_table must be [B][width]")
        B, width = (int(x) for x in self.block_table.shape)
        _check_dev(self.block_table, "block_table", torch.int32)
        index = self.block_table.get_device()
        for n in ("lens", "held"):
            _flat(getattr(self, n), n, torch.int32, B, index)
        if self.free.dim() != 1 or self.free.numel() < 2:
            raise ValueError("free must be [2 + pool]")
        _flat(self.free, "free", torch.int32, self.free.numel(), index)
        desc = _KVPagesDesc(B, width, self.page_size, self.free.numel() - 2, _dptr(self.block_table), _dptr(self.lens),
                            _dptr(self.held), _dptr(self.free))
        for name, value in (("sequences", B), ("width", width), ("device", self.block_table.device),
                            ("_index", index), ("_desc", desc), ("_ref", ctypes.addressof(desc)),
                            ("_at", self._addresses())):
            object.__setattr__(self, name, value)

    def _addresses(self):
        return (self.block_table.data_ptr(), self.lens.data_ptr(), self.held.data_ptr(), self.free.data_ptr())

    def _pointer(self):
        """The descriptor; a tensor given another storage is taken up, and checked, by the next call."""
        if self._addresses() != self._at:
            self.__post_init__()
        return self._ref


def new_kv_pages(sequences: int, width: int, num_pages: int, page_size: int, device="cuda") -> KVPages:
    """Empty sequences, and all of a cache's num_pages pages free (page 0 is taken first)."""
    import torch

    def zeros(*shape):
        return torch.zeros(shape, dtype=torch.int32, device=device)

    free = zeros(2 + num_pages)
    free[0] = num_pages
    free[2:] = torch.arange(num_pages - 1, -1, -1, dtype=torch.int32, device=device)
    return KVPages(zeros(sequences, width), zeros(sequences), zeros(sequences), free, page_size)


class KVStep(NamedTuple):
    """What a step's calls take: slots int64 [rows] (kv_append, qk_norm_rope_append), positions int32 [rows],
    sequences int32 [rows] (-1: no sequence's), q_start int32 [B + 1] and kv_lens int32 [B] (attention_tree)."""
    slots: "object"
    positions: "object"
    sequences: "object"
    q_start: "object"
    kv_lens: "object"


def kv_step(pages: KVPages, keep, new_tokens, rows: int, tree_mask=None, out: Optional[KVStep] = None,
            stream=None) -> KVStep:
    """One step of all sequences, on the GPU: sequence b keeps the first keep[b] of its tokens (int32 [B]; None: all
    of them) and appends new_tokens[b] (int32 [B]), in rows q_start[b] up to q_start[b + 1] of the step's `rows` token
    rows. Pages that are no longer needed go back, those needed are taken; block_table, lens, held and free are
    updated in place. tree_mask: int64 [rows], attention_tree's: positions follow the depth in the tree. A sequence
    whose pages (or rows) do not fit waits: its slots are -1 and its kv_lens 0, and it keeps its kept tokens. Rows behind
    the last sequence get slot -1, position 0, sequence -1. out: tensors for the
    results, over none of the call's inputs or pages (refused otherwise)."""
    import torch
    ref, i32 = pages._pointer(), torch.int32
    index, B = pages._index, pages.sequences
    if out is None:
        dev = pages.device
        out = KVStep(_new_output((rows,), torch.int64, dev, stream), _new_output((rows,), i32, dev, stream),
                     _new_output((rows,), i32, dev, stream), _new_output((B + 1,), i32, dev, stream),
                     _new_output((B,), i32, dev, stream))
    slots, positions, sequences, q_start, kv_lens = out
    rc = _launch(
        load_library().kv_pages_step, index, stream, ref,
        None if keep is None else _flat(keep, "keep", i32, B, index), _flat(new_tokens, "new_tokens", i32, B, index),
        None if tree_mask is None else _flat(tree_mask, "tree_mask", torch.int64, rows, index), rows,
        _flat(slots, "slots", torch.int64, rows, index), _flat(positions, "positions", i32, rows, index),
        _flat(sequences, "sequences", i32, rows, index), _flat(q_start, "q_start", i32, B + 1, index),
        _flat(kv_lens, "kv_lens", i32, B, index))
    _check(rc, "kv_pages_step")
    return out


# ---- query and key heads normed, rotated, and written to the cache ----

# bsp_rotation of include/bitmap_spmm.h, packed: a call's descriptors are bytes (a ctypes structure takes three times as long)
_ROTATION = struct.Struct("@qiPPPPf4x")


def rope_frequencies(rot: int, base: float = 10000.0, angles=None, device="cuda"):
    """int64 [rot / 2]: the turn of each pair per position, as a fraction of 2^64 of a whole one. angles: radians per
    position (float64 [rot / 2], for scaled forms); default base ** (-2 i / rot)."""
    import torch
    if angles is None:
        angles = float(base) ** (-2.0 * np.arange(rot // 2) / max(rot, 1))
    angles = np.asarray(angles, np.float64)
    if angles.shape != (rot // 2,) or not np.isfinite(angles).all():
        raise ValueError("angles must be rot / 2 finite radians per position")
    turns = np.mod(angles / (2.0 * np.pi), 1.0)
    # 2^64 turns in two 32-bit halves, each an exact product
    hi = np.floor(turns * 2.0 ** 32)
    lo = np.floor((turns * 2.0 ** 32 - hi) * 2.0 ** 32)
    words = (hi.astype(np.uint64) << np.uint64(32)) | lo.astype(np.uint64)
    return torch.from_numpy(words.view(np.int64)).to(device)


def _rotation(positions, freq, q_weight, k_weight, eps, interleaved, n, dim, index) -> bytes:
    import torch
    f16 = torch.float16
    rot = f = p = 0
    if freq is not None:
        rot = 2 * freq.numel()
        f = _flat(freq, "freq", torch.int64, rot // 2, index)
        p = _flat(positions, "positions", torch.int32, n, index)
    return _ROTATION.pack(rot, 1 if interleaved else 0, f, p,
                          0 if q_weight is None else _flat(q_weight, "q_weight", f16, dim, index),
                          0 if k_weight is None else _flat(k_weight, "k_weight", f16, dim, index), eps)


def _heads(t, name):
    if t.dim() != 3 or not t.is_cuda:
        raise ValueError(f"{name} must be [tokens][heads][head_dim] on the device")
    return t.shape


def qk_norm_rope(Q, K, positions, freq, q_weight=None, k_weight=None, eps: float = 1e-6, interleaved: bool = False,
                 Qo=None, Ko=None, stream=None):
    """Queries and keys normed head by head (x / sqrt(mean(x^2) + eps) * weight; no weight: not normed) and rotated to
    their positions (int32 [n]): Q float16 [n][q_heads][head_dim], K [n][kv_heads][head_dim], a token's heads contiguous.
    freq: rope_frequencies(rot), rot <= head_dim a multiple of 16 (None: no rotation). Qo, Ko: the results (may be
    Q, K)."""
    import torch
    n, hq, dim = _heads(Q, "Q")
    hkv = _heads(K, "K")[1]
    index = Q.get_device()
    qs, ks = _rows(Q, "Q", n, hq, dim, index), _rows(K, "K", n, hkv, dim, index)
    if Qo is None:
        Qo, qo = _new_output((n, hq, dim), torch.float16, Q.device, stream), hq * dim
    else:
        qo = _rows(Qo, "Qo", n, hq, dim, index)
    if Ko is None:
        Ko, ko = _new_output((n, hkv, dim), torch.float16, Q.device, stream), hkv * dim
    else:
        ko = _rows(Ko, "Ko", n, hkv, dim, index)
    d = _rotation(positions, freq, q_weight, k_weight, eps, interleaved, n, dim, index)
    rc = _launch(load_library().qk_norm_rope_f16, index, stream, Q.data_ptr(), qs, K.data_ptr(), ks, n, hq, hkv, dim,
                 d, Qo.data_ptr(), qo, Ko.data_ptr(), ko)
    _check(rc, "qk_norm_rope_f16")
    return Qo, Ko


def qk_norm_rope_append(Q, K, V, positions, freq, cache: KVCache, slots, q_weight=None, k_weight=None,
                        eps: float = 1e-6, interleaved: bool = False, Qo=None, stream=None):
    """qk_norm_rope with the keys and the values V written to the cache's slots (int64 [n]) in the same pass: what
    qk_norm_rope and kv_append leave there, bit for bit. Returns the queries."""
    import torch
    n, hq, _ = _heads(Q, "Q")
    hkv, dim, index = cache.kv_heads, cache.head_dim, cache._index
    qs, ks, vs = _rows(Q, "Q", n, hq, dim, index), _rows(K, "K", n, hkv, dim, index), _rows(V, "V", n, hkv, dim, index)
    if Qo is None:
        Qo, qo = _new_output((n, hq, dim), torch.float16, cache.device, stream), hq * dim
    else:
        qo = _rows(Qo, "Qo", n, hq, dim, index)
    d = _rotation(positions, freq, q_weight, k_weight, eps, interleaved, n, dim, index)
    rc = _launch(load_library().qk_norm_rope_append_f16, index, stream, Q.data_ptr(), qs, K.data_ptr(), ks,
                 V.data_ptr(), vs, n, hq, d, cache._ref, _flat(slots, "slots", torch.int64, n, index),
                 Qo.data_ptr(), qo)
    _check(rc, "qk_norm_rope_append_f16")
    return Qo


# ---- hidden states quantised token by token ----

# bsp_tokens of include/bitmap_spmm.h, packed
_TOKENS = struct.Struct("@qqPqPqPf4xPqPqP")


class Tokens(NamedTuple):
    """Quantised tokens: codes (INT8: int8 [n][K], rows of whole 16 bytes; INT4: uint8 [n][ceil(K / 2)], packed), scale
    float32 [n], and where asked for x16 (float16 [n][K], the values before quantisation) and hidden (float16 [n][K],
    the residual sum)."""
    codes: "object"
    scale: "object"
    x16: "object" = None
    hidden: "object" = None


def _matrix_rows(t, name, dtype, n, width, index) -> int:
    """Check an [n][width] tensor whose rows may be strided; returns the stride between rows."""
    import torch
    # the common case in few steps; what is wrong is named below
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index and t.shape == (n, width):
        if t.is_contiguous():
            return width
        s0, s1 = t.stride()
        if s1 == 1 or width <= 1:
            if n <= 1:
                return width
            if s0 >= width:
                return s0
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on device {index}")
    raise ValueError(f"{name} must be [{n}][{width}] with contiguous rows that do not overlap, got {tuple(t.shape)}")


def _code_rows(codes, dtype, n, K, index):
    """(address, row stride) of codes as Tokens holds them."""
    import torch
    if dtype == INT8:
        return codes.data_ptr(), _matrix_rows(codes, "codes", torch.int8, n, K, index)
    if dtype == INT4:
        return codes.data_ptr(), _matrix_rows(codes, "codes", torch.uint8, n, (K + 1) // 2, index)
    raise ValueError("codes are INT8 or INT4")


def quantize_tokens(X, dtype: int, weight=None, eps: float = 1e-6, residual=None, hidden=None, x16=None, codes=None,
                    scale=None, stream=None) -> Tokens:
    """Tokens X float16 [n][K] as INT8 or (packed) INT4 codes with one scale each, for gemm_w8a8 and spmm_w4a4_dq.
    residual: float16 [n][K], added first (the sum, rounded to float16, goes to `hidden`, which may be X or residual).
    weight: float16 [K], the tokens are normed first (x / sqrt(mean(x^2) + eps) * weight). x16: True or a tensor for the
    float16 values that the codes quantise. Every code is the correctly rounded one."""
    import torch
    if X.dim() != 2 or not X.is_cuda or X.shape[1] == 0:
        raise ValueError("X must be [n][K] on the device, K > 0")
    n, K = X.shape
    index, f16, dev = X.get_device(), torch.float16, X.device
    xs = _matrix_rows(X, "X", f16, n, K, index)
    if codes is None and dtype == INT8:
        cs = (K + 15) // 16 * 16
        codes = _new_output((n, cs), torch.int8, dev, stream)
        cp = codes.data_ptr()
        if cs != K:
            codes = codes[:, :K]
    elif codes is None and dtype == INT4:
        cs = (K + 1) // 2
        codes = _new_output((n, cs), torch.uint8, dev, stream)
        cp = codes.data_ptr()
    else:
        cp, cs = _code_rows(codes, dtype, n, K, index)
    if scale is None:
        scale = _new_output((n,), torch.float32, dev, stream)
        sp = scale.data_ptr()
    else:
        sp = _flat(scale, "scale", torch.float32, n, index)
    r = rs = h = hs = x = x16s = 0
    if residual is not None:
        rs, hs = _matrix_rows(residual, "residual", f16, n, K, index), K
        if hidden is None:
            hidden = _new_output((n, K), f16, dev, stream)
        else:
            hs = _matrix_rows(hidden, "hidden", f16, n, K, index)
        r, h = residual.data_ptr(), hidden.data_ptr()
    elif hidden is not None:
        raise ValueError("hidden goes with residual")
    if x16 is True:
        x16 = _new_output((n, K), f16, dev, stream)
    elif x16 is False:
        x16 = None
    if x16 is not None:
        x16s = _matrix_rows(x16, "x16", f16, n, K, index)
        x = x16.data_ptr()
    d = _TOKENS.pack(n, K, X.data_ptr(), xs, r, rs, 0 if weight is None else _flat(weight, "weight", f16, K, index), eps,
                     h, hs, x, x16s, sp)
    rc = _launch(load_library().quantize_tokens_f16, index, stream, d, dtype, cp, cs)
    _check(rc, "quantize_tokens_f16")
    return Tokens(codes, scale, x16, hidden)


def dequantize_tokens(codes, scale, dtype: int, K: int, X=None, stream=None):
    """float16 X [n][K], the values that the codes of quantize_tokens stand for."""
    import torch
    if not scale.is_cuda:
        raise TypeError("scale must be a CUDA (HIP) tensor")
    n, index = scale.numel(), scale.get_device()
    sp = _flat(scale, "scale", torch.float32, n, index)
    cp, cs = _code_rows(codes, dtype, n, K, index)
    if X is None:
        X, xs = _new_output((n, K), torch.float16, scale.device, stream), K
    else:
        xs = _matrix_rows(X, "X", torch.float16, n, K, index)
    rc = _launch(load_library().dequantize_tokens_f16, index, stream, cp, cs, dtype, sp, n, K, X.data_ptr(), xs)
    _check(rc, "dequantize_tokens_f16")
    return X


# ---- dense 8-bit product ----

@dataclass
class EncodedInt8:
    """A dense int8 matrix laid out for gemm_w8a8 (host): tiles uint8, scale float32 [M]."""
    M: int
    K: int
    tiles: np.ndarray
    scale: np.ndarray

    def to_device(self, device="cuda") -> "DenseInt8":
        import torch
        return DenseInt8(self.M, self.K, torch.from_numpy(self.tiles).to(device),
                         torch.from_numpy(self.scale).to(device))


@dataclass(frozen=True)
class DenseInt8:
    """A dense int8 matrix in device memory, as encode_int8 laid it out, with the scale of each row (channel)."""
    M: int
    K: int
    tiles: "object"
    scale: "object"

    def __post_init__(self):
        import torch
        _check_dev(self.tiles, "tiles", torch.uint8, (self.M + 15) // 16 * ((self.K + 63) // 64) * 1024)
        index = self.tiles.get_device()
        _flat(self.scale, "scale", torch.float32, self.M, index)
        object.__setattr__(self, "_index", index)
        object.__setattr__(self, "_at", (self.tiles.data_ptr(), self.scale.data_ptr()))

    def _pointers(self):
        """Where the tensors lie; one given another storage is taken up, and checked, by the next call."""
        if (self.tiles.data_ptr(), self.scale.data_ptr()) != self._at:
            self.__post_init__()
        return self._at


def encode_int8(W: np.ndarray, scale: np.ndarray) -> EncodedInt8:
    """Lay out a dense host matrix, int8 [M][K] with float32 [M] scales, for gemm_w8a8."""
    L = load_library()
    if W.dtype != np.int8 or W.ndim != 2:
        raise TypeError("W must be a 2-D int8 array")
    W = np.ascontiguousarray(W)
    M, K = W.shape
    scale = np.ascontiguousarray(scale, np.float32)
    if scale.shape != (M,):
        raise ValueError("scale must be [M]")
    tiles = np.empty(max(L.int8_tiles_bytes(M, K), 0), np.uint8)
    _check(L.encode_int8_tiles(_np_ptr(W), M, K, K, _np_ptr(tiles)), "encode_int8_tiles")
    return EncodedInt8(M, K, tiles, scale)


def gemm_workspace_bytes(M: int, K: int, N: int) -> int:
    """Bytes of workspace gemm_w8a8 uses to split K over workgroups, for any number of tokens up to N (0: none)."""
    out = ctypes.c_int64(0)
    _check(load_library().gemm_w8a8_workspace_bytes(M, K, N, ctypes.byref(out)), "gemm_w8a8_workspace_bytes")
    return int(out.value)


def new_gemm_workspace(W: DenseInt8, N: int, device="cuda"):
    """A zero-filled workspace for gemm_w8a8 with up to N tokens (None if none is used).
    It is cleared on the current stream: calls on another one wait for that."""
    import torch
    n = gemm_workspace_bytes(W.M, W.K, N)
    return torch.zeros(n, dtype=torch.uint8, device=device) if n else None


def describe_gemm(M: int, K: int, N: int, workspace: bool = False) -> str:
    """The kernel, tile (channels x tokens) and split of K that gemm_w8a8 takes."""
    buf = ctypes.create_string_buffer(256)
    _check(load_library().gemm_w8a8_describe(M, K, N, int(workspace), buf, 256), "gemm_w8a8_describe")
    return buf.value.decode()


def gemm_w8a8(W: DenseInt8, X, scale_x, Y=None, workspace=None, stream=None):
    """float16 Y [N][M] = (W x_n) * W.scale[m] * scale_x[n], int32 sums, any N. X: int8 [N][K], rows of whole 16 bytes
    in memory (as quantize_tokens leaves them); scale_x: float32 [N]. workspace: new_gemm_workspace of W and as
    many tokens or more, or None for no split over K; calls that share one must be ordered."""
    import torch
    if X.dim() != 2 or X.shape[1] != W.K:
        raise ValueError("X must be [N][K]")
    tiles, scale_w = W._pointers()
    N, M, K, index = X.shape[0], W.M, W.K, W._index
    xs = _matrix_rows(X, "X", torch.int8, N, K, index)
    if N <= 1 or K == 0:
        xs = (K + 15) // 16 * 16
    if xs != K and N > 0 and X.untyped_storage().nbytes() < X.storage_offset() + N * xs:
        raise ValueError("X: every row must be readable up to its stride")
    if Y is None:
        Y, ys = _new_output((N, M), torch.float16, X.device, stream), M
    else:
        ys = _matrix_rows(Y, "Y", torch.float16, N, M, index)
    wp, wb = (None, 0) if workspace is None else _ws_args(workspace, index)
    rc = _launch(load_library().gemm_w8a8_dq, index, stream, tiles, M, K, X.data_ptr(), xs, N, scale_w,
                 _flat(scale_x, "scale_x", torch.float32, N, index), Y.data_ptr(), ys, wp, wb)
    _check(rc, "gemm_w8a8_dq")
    return Y
