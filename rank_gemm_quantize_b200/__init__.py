"""Python binding of the SVDQuant W4A4 + low-rank linear layer for B200 (sm_100a).

Argument marshalling only: every step of the layer runs in the CUDA kernels of
``libsvdq.so`` (built in-tree by ``rank_gemm_quantize_b200.build``), reached
through the C ABI declared in ``include/svdq.h``. PyTorch is used for device
memory and the current CUDA stream; there is no CPU or PyTorch fallback -
importing this module without the built library raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
from dataclasses import dataclass
from enum import IntEnum
from typing import Optional

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsvdq.so")

INT4_G64 = "int4_g64"
NVFP4_G16 = "nvfp4_g16"
_FMT = {INT4_G64: 0, NVFP4_G16: 1}
_FMT_NAME = {0: INT4_G64, 1: NVFP4_G16}


class Status(IntEnum):
    OK = 0
    INVALID_ARG = 1
    UNSUPPORTED = 2
    OOM = 3
    CUDA = 4
    NUMERIC = 5
    DEVICE_TIMEOUT = 6


class SvdqError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{Status(status).name}: {message}")
        self.status = Status(status)


NO_SMOOTHING = 1  # svdq_config.flags: s = 1 for every channel
MAX_ADAPTERS = 8


class _Config(ctypes.Structure):
    _fields_ = [("K", ctypes.c_int), ("N", ctypes.c_int), ("rank", ctypes.c_int), ("alpha", ctypes.c_float),
                ("s_min", ctypes.c_float), ("fmt", ctypes.c_int), ("flags", ctypes.c_uint)]


class _Info(ctypes.Structure):
    _fields_ = [("K", ctypes.c_int), ("N", ctypes.c_int), ("rank", ctypes.c_int), ("rank_pad", ctypes.c_int),
                ("fmt", ctypes.c_int), ("alpha", ctypes.c_float), ("g_x", ctypes.c_float), ("g_w", ctypes.c_float),
                ("t_scale", ctypes.c_float), ("base_rank", ctypes.c_int), ("flags", ctypes.c_uint),
                ("adapter_slots", ctypes.c_uint), ("adapter_col_start", ctypes.c_int * (MAX_ADAPTERS + 1))]


class _BlobHeader(ctypes.Structure):
    _fields_ = [("magic", ctypes.c_uint32), ("version", ctypes.c_uint32), ("fmt", ctypes.c_int32),
                ("K", ctypes.c_int32), ("N", ctypes.c_int32), ("rank", ctypes.c_int32), ("alpha", ctypes.c_float),
                ("g_x", ctypes.c_float), ("g_w", ctypes.c_float), ("reserved", ctypes.c_float),
                ("off_s", ctypes.c_uint64), ("off_inv_s", ctypes.c_uint64), ("off_L1", ctypes.c_uint64),
                ("off_L2", ctypes.c_uint64), ("off_codes", ctypes.c_uint64), ("off_scales", ctypes.c_uint64),
                ("off_bias", ctypes.c_uint64), ("total", ctypes.c_uint64)]


class _Attention(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("batch", ctypes.c_int), ("q_rows", ctypes.c_int), ("k_rows", ctypes.c_int),
                ("q_heads", ctypes.c_int), ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("causal", ctypes.c_int), ("scale", ctypes.c_float)] + [
                    (f"{t}_{a}_stride", ctypes.c_longlong) for t in "qkv" for a in ("row", "head")] + [
                        (n, ctypes.c_void_p) for n in ("q", "k", "v", "q_offsets", "k_offsets", "out", "workspace")] + [
                            ("workspace_bytes", ctypes.c_ulonglong)]


class _DenseLinear(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("dtype", "activation", "M", "K", "N")] + [
        (n, ctypes.c_void_p) for n in ("X", "W", "bias", "residual", "Y")]


class _ResidualNorm(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("dtype", "x_dtype", "rows", "dim", "seqs", "post_norm", "norm")] + [
        (n, ctypes.c_float) for n in ("residual_scale", "eps")] + [
            (n, ctypes.c_void_p) for n in ("x", "y", "x_out", "h_out", "gate", "post_weight", "post_bias", "weight",
                                           "bias", "scale", "shift", "offsets")]


def _packer(cls):
    """Packs a call's arguments as the C struct, without the cost of a ctypes object (0 for NULL)."""
    code = {ctypes.c_int: "i", ctypes.c_float: "f", ctypes.c_void_p: "P", ctypes.c_longlong: "q", ctypes.c_ulonglong: "Q"}
    return struct.Struct("@" + "".join(code[t] for _, t in cls._fields_)).pack


_pack_attention, _pack_dense_linear, _pack_residual_norm = map(_packer, (_Attention, _DenseLinear, _ResidualNorm))

# Every symbol include/svdq.h declares, with its ctypes signature.
_VP, _I, _F, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
SIGNATURES = {
    "svdq_calibrate_absmax": [_VP, _I, _I, _VP, _VP],
    "svdq_prepare_weights": [ctypes.POINTER(_Config), _VP, _VP, _VP, _VP, ctypes.POINTER(_VP)],
    "svdq_prepare_weights_with_factors": [ctypes.POINTER(_Config), _VP, _VP, _VP, _VP, _VP, _VP, ctypes.POINTER(_VP)],
    "svdq_workspace_size": [_VP, _I, ctypes.POINTER(_SZ)],
    "svdq_linear_forward": [_VP, _VP, _I, _VP, _VP, _SZ, _VP],
    "svdq_linear_forward_profiled": [_VP, _VP, _I, _VP, _VP, _SZ, _VP, ctypes.POINTER(_VP)],
    "svdq_linear_forward_noalloc": [_VP, _VP, _I, _VP, _VP],
    "svdq_linear_forward_masked": [_VP, _VP, _I, _VP, _VP, _SZ, _VP, _VP],
    "svdq_attach_lora": [_VP, _VP, _VP, _I, _F, _VP, ctypes.POINTER(_I)],
    "svdq_detach_lora": [_VP, _I, _VP],
    "svdq_quantize_activations": [_VP, _VP, _I, _VP, _VP, _VP, _VP],
    "svdq_export_weights": [_VP, _VP, ctypes.POINTER(_SZ), _VP],
    "svdq_layer_get_info": [_VP, ctypes.POINTER(_Info)],
    "svdq_device_status": [_VP, _VP],
    "svdq_destroy": [_VP],
    "svdq_last_error": [],
    "svdq_selftest_bounded_wait": [ctypes.c_ulonglong, _VP],
    "svdq_debug_fail_allocation": [ctypes.c_longlong],
    "svdq_mlp_workspace_size": [_VP, _VP, _I, ctypes.POINTER(_SZ)],
    "svdq_mlp_workspace_layout": [_VP, _VP, _I, ctypes.POINTER(_SZ)],
    "svdq_mlp_forward": [_VP, _VP, _VP, _I, _VP, _VP, _SZ, _VP],
    "svdq_mlp_forward_profiled": [_VP, _VP, _VP, _I, _VP, _VP, _SZ, _VP, ctypes.POINTER(_VP)],
    "svdq_w4a16_prepare": [_VP, _VP, _I, _I, _VP, ctypes.POINTER(_VP)],
    "svdq_w4a16_forward": [_VP, _VP, _I, _VP, _VP],
    "svdq_w4a16_export": [_VP, _VP, _VP, _VP],
    "svdq_w4a16_destroy": [_VP],
    "svdq_attention_workspace_size": [_VP, ctypes.POINTER(_SZ)],
    "svdq_attention_forward": [_VP, _VP],
    "svdq_dense_linear_forward": [_VP, _VP],
    "svdq_residual_norm": [_VP, _VP],
    "svdq_operator_status": [_VP],
    "svdq_selftest_operator_wait": [_I, _VP],
}


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Loads libsvdq.so and declares its C ABI. Raises if it is missing."""
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python -m rank_gemm_quantize_b200.build`")
    lib = ctypes.CDLL(path)
    for name, args in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = {"svdq_last_error": ctypes.c_char_p, "svdq_debug_fail_allocation": None}.get(name, ctypes.c_int)
    return lib


_lib: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        _lib = load_library()
    return _lib


def _check(status: int) -> None:
    if status != 0:
        raise SvdqError(status, lib().svdq_last_error().decode())


def _stream(stream=None) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("tensors must be contiguous CUDA tensors")
    return t.data_ptr()


def calibrate_absmax(X: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """A_scale (per input channel absolute maximum) folded into `out` (float32 [K])."""
    M, K = X.shape
    if out is None:
        out = torch.zeros(K, dtype=torch.float32, device=X.device)
    _check(lib().svdq_calibrate_absmax(_ptr(X), M, K, _ptr(out), _stream(stream)))
    return out


def selftest_bounded_wait(limit_ns: int = 50_000_000, stream=None) -> Status:
    st = lib().svdq_selftest_bounded_wait(limit_ns, _stream(stream))
    return Status(st)


@dataclass
class LayerInfo:
    K: int
    N: int
    rank: int
    rank_pad: int
    fmt: str
    alpha: float
    g_x: float
    g_w: float
    t_scale: float
    base_rank: int = 0
    flags: int = 0
    adapter_slots: int = 0
    adapter_col_start: tuple = ()


class Layer:
    """A prepared SVDQuant linear layer (owns its device buffers)."""

    def __init__(self, handle: int, device: Optional[torch.device] = None):
        self._h = ctypes.c_void_p(handle)
        self._ws: Optional[torch.Tensor] = None
        self._info: Optional[LayerInfo] = None
        self.device = torch.device("cuda", torch.cuda.current_device()) if device is None else device

    @classmethod
    def prepare(cls, W: torch.Tensor, bias: Optional[torch.Tensor], act_absmax: torch.Tensor, fmt: str, rank: int,
                alpha: float = 0.5, s_min: float = 1e-5, factors=None, smooth: bool = True, stream=None) -> "Layer":
        """Offline preparation; rank 0 gives the smoothing-only layer, smooth=False
        keeps s = 1 (both ablations of the method)."""
        K, N = W.shape
        cfg = _Config(K, N, rank, alpha, s_min, _FMT[fmt], 0 if smooth else NO_SMOOTHING)
        out = ctypes.c_void_p()
        if factors is None:
            st = lib().svdq_prepare_weights(ctypes.byref(cfg), _ptr(W), _ptr(bias), _ptr(act_absmax), _stream(stream),
                                            ctypes.byref(out))
        else:
            L1, L2 = factors
            st = lib().svdq_prepare_weights_with_factors(ctypes.byref(cfg), _ptr(W), _ptr(bias), _ptr(act_absmax),
                                                         _ptr(L1), _ptr(L2), _stream(stream), ctypes.byref(out))
        _check(st)
        return cls(out.value, W.device)

    def info(self) -> LayerInfo:
        if self._info is None:
            i = _Info()
            _check(lib().svdq_layer_get_info(self._h, ctypes.byref(i)))
            self._info = LayerInfo(i.K, i.N, i.rank, i.rank_pad, _FMT_NAME[i.fmt], i.alpha, i.g_x, i.g_w, i.t_scale,
                                   i.base_rank, i.flags, i.adapter_slots, tuple(i.adapter_col_start))
        return self._info

    def workspace_size(self, M: int) -> int:
        n = ctypes.c_size_t()
        _check(lib().svdq_workspace_size(self._h, M, ctypes.byref(n)))
        return n.value

    def _check_io(self, X: torch.Tensor, out: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None) -> int:
        """The shapes, dtypes and placement the C ABI assumes; the library reads
        X through a tensor map built from the layer's K, so a narrower or
        strided X would be read past its end."""
        info = self.info()
        if X.dim() != 2 or X.shape[1] != info.K:
            raise ValueError(f"X must be [M, {info.K}], got {tuple(X.shape)}")
        if X.dtype != torch.bfloat16 or not X.is_contiguous():
            raise ValueError("X must be a contiguous bfloat16 tensor")
        if X.device != self.device:
            raise ValueError(f"X is on {X.device}, the layer on {self.device}")
        if out is not None:
            if tuple(out.shape) != (X.shape[0], info.N) or out.dtype != torch.bfloat16 or not out.is_contiguous():
                raise ValueError(f"out must be a contiguous bfloat16 [{X.shape[0]}, {info.N}] tensor")
            if out.device != self.device:
                raise ValueError(f"out is on {out.device}, the layer on {self.device}")
        if workspace is not None:
            if workspace.dtype != torch.uint8 or not workspace.is_contiguous() or workspace.device != self.device:
                raise ValueError("workspace must be a contiguous uint8 tensor on the layer's device")
        return info.N

    def workspace(self, M: int, device=None) -> torch.Tensor:
        need = self.workspace_size(M)
        if self._ws is None or self._ws.numel() < need:
            self._ws = torch.empty(need, dtype=torch.uint8, device=device or "cuda")
        return self._ws

    def forward(self, X: torch.Tensor, out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
        N = self._check_io(X, out, workspace)
        M = X.shape[0]
        if out is None:
            out = torch.empty(M, N, dtype=torch.bfloat16, device=X.device)
        ws = workspace if workspace is not None else self.workspace(M, X.device)
        _check(lib().svdq_linear_forward(self._h, _ptr(X), M, _ptr(out), _ptr(ws), ws.numel(), _stream(stream)))
        return out

    __call__ = forward

    def forward_noalloc(self, X: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """forward() on the library's fixed scratch array (no workspace, no allocation by the library)."""
        N = self._check_io(X, out)
        M = X.shape[0]
        if out is None:
            out = torch.empty(M, N, dtype=torch.bfloat16, device=X.device)
        _check(lib().svdq_linear_forward_noalloc(self._h, _ptr(X), M, _ptr(out), _stream(stream)))
        return out

    def forward_profiled(self, X: torch.Tensor, out: torch.Tensor, workspace: torch.Tensor, events, stream=None):
        """forward() recording three torch.cuda.Event objects around its two kernels."""
        self._check_io(X, out, workspace)
        arr = (ctypes.c_void_p * 3)(*[e.cuda_event for e in events])
        _check(lib().svdq_linear_forward_profiled(self._h, _ptr(X), X.shape[0], _ptr(out), _ptr(workspace),
                                                  workspace.numel(), _stream(stream), arr))
        return out

    def quantize_activations(self, X: torch.Tensor, stream=None):
        """(codes, scales, T) of the activation kernel in its documented layouts."""
        info = self.info()
        M, K = X.shape
        M_pad = (M + 127) // 128 * 128
        dev = X.device
        if info.fmt == INT4_G64:
            codes = torch.empty(M_pad, K, dtype=torch.uint8, device=dev)
            scales = torch.empty(K // 64, M_pad, dtype=torch.float32, device=dev)
        else:
            codes = torch.empty(M_pad, K // 2, dtype=torch.uint8, device=dev)
            scales = torch.empty(M_pad // 128 * (K // 64) * 512, dtype=torch.uint8, device=dev)
        T = torch.empty(M_pad, info.rank_pad, dtype=torch.bfloat16, device=dev)
        _check(lib().svdq_quantize_activations(self._h, _ptr(X), M, _ptr(codes), _ptr(scales),
                                               _ptr(T) if info.rank_pad else None, _stream(stream)))
        return codes, scales, T

    def attach_lora(self, A: torch.Tensor, B: torch.Tensor, scale: float = 1.0, stream=None) -> int:
        """Adds scale * X A B to the branch; returns the adapter's slot."""
        self._info = None
        slot = ctypes.c_int(-1)
        _check(lib().svdq_attach_lora(self._h, _ptr(A), _ptr(B), A.shape[1], scale, _stream(stream),
                                      ctypes.byref(slot)))
        return slot.value

    def detach_lora(self, slot: int, stream=None) -> None:
        """Removes the adapter in `slot` (the branch returns to what it was without it)."""
        self._info = None
        _check(lib().svdq_detach_lora(self._h, slot, _stream(stream)))

    def forward_masked(self, X: torch.Tensor, row_adapter_mask: torch.Tensor, out: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """forward() where row m uses the adapters whose slot bits are set in
        row_adapter_mask[m] (int32/uint32 [M] on the layer's device)."""
        N = self._check_io(X, out, workspace)
        M = X.shape[0]
        if (row_adapter_mask.dim() != 1 or row_adapter_mask.shape[0] != M or row_adapter_mask.element_size() != 4
                or row_adapter_mask.device != self.device or not row_adapter_mask.is_contiguous()):
            raise ValueError("row_adapter_mask must be a contiguous 32-bit [M] tensor on the layer's device")
        if out is None:
            out = torch.empty(M, N, dtype=torch.bfloat16, device=X.device)
        ws = workspace if workspace is not None else self.workspace(M, X.device)
        _check(lib().svdq_linear_forward_masked(self._h, _ptr(X), M, _ptr(out), _ptr(ws), ws.numel(),
                                                _ptr(row_adapter_mask), _stream(stream)))
        return out

    def export(self, stream=None) -> dict:
        """Canonical prepared weights (numpy arrays)."""
        n = ctypes.c_size_t()
        _check(lib().svdq_export_weights(self._h, None, ctypes.byref(n), _stream(stream)))
        buf = (ctypes.c_uint8 * n.value)()
        _check(lib().svdq_export_weights(self._h, ctypes.cast(buf, ctypes.c_void_p), ctypes.byref(n), _stream(stream)))
        raw = np.frombuffer(buf, dtype=np.uint8).copy()
        hd = _BlobHeader.from_buffer_copy(raw[:ctypes.sizeof(_BlobHeader)].tobytes())
        K, N, r = hd.K, hd.N, hd.rank

        def sec(off, dtype, shape):
            cnt = int(np.prod(shape))
            return raw[off:off + cnt * np.dtype(dtype).itemsize].view(dtype).reshape(shape).copy()

        bf = lambda a: (a.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
        out = {
            "fmt": _FMT_NAME[hd.fmt], "K": K, "N": N, "rank": r, "alpha": hd.alpha,
            "g_x": np.float32(hd.g_x), "g_w": np.float32(hd.g_w),
            "s": sec(hd.off_s, np.float32, (K,)), "inv_s": sec(hd.off_inv_s, np.float32, (K,)),
            "L1": bf(sec(hd.off_L1, np.uint16, (K, r))), "L2": bf(sec(hd.off_L2, np.uint16, (r, N))),
            "codes_packed": sec(hd.off_codes, np.uint8, (N, K // 2)),
            "bias": bf(sec(hd.off_bias, np.uint16, (N,))),
        }
        if hd.fmt == 0:
            out["scales"] = sec(hd.off_scales, np.float32, (N, K // 64))
        else:
            out["scales"] = sec(hd.off_scales, np.uint8, (N, K // 16))
        return out

    def device_status(self, stream=None) -> Status:
        return Status(lib().svdq_device_status(self._h, _stream(stream)))

    def close(self) -> None:
        if self._h is not None and self._h.value:
            lib().svdq_destroy(self._h)
        self._h = None
        self._ws = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class WeightOnlyLayer:
    """The 4-bit weight-only (W4A16) baseline: INT4 group-64 weights, bf16
    activations, dequantized on chip (include/svdq.h, svdq_w4a16_*)."""

    def __init__(self, W: torch.Tensor, bias: Optional[torch.Tensor] = None, stream=None):
        if W.dim() != 2 or W.dtype != torch.bfloat16 or not W.is_cuda or not W.is_contiguous():
            raise ValueError("W must be a contiguous bfloat16 CUDA tensor [K, N]")
        self.K, self.N = W.shape
        self.device = W.device
        out = ctypes.c_void_p()
        _check(lib().svdq_w4a16_prepare(_ptr(W), _ptr(bias), self.K, self.N, _stream(stream), ctypes.byref(out)))
        self._h = out

    def forward(self, X: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        if X.dim() != 2 or X.shape[1] != self.K or X.dtype != torch.bfloat16 or not X.is_contiguous() \
                or X.device != self.device:
            raise ValueError(f"X must be a contiguous bfloat16 [M, {self.K}] tensor on {self.device}")
        M = X.shape[0]
        if out is None:
            out = torch.empty(M, self.N, dtype=torch.bfloat16, device=X.device)
        elif tuple(out.shape) != (M, self.N) or out.dtype != torch.bfloat16 or not out.is_contiguous():
            raise ValueError(f"out must be a contiguous bfloat16 [{M}, {self.N}] tensor")
        _check(lib().svdq_w4a16_forward(self._h, _ptr(X), M, _ptr(out), _stream(stream)))
        return out

    __call__ = forward

    def export(self, stream=None):
        """(codes uint8 [N, K/2] packed nibbles, scales float32 [K/64, N])."""
        codes = np.zeros((self.N, self.K // 2), dtype=np.uint8)
        scales = np.zeros((self.K // 64, self.N), dtype=np.float32)
        _check(lib().svdq_w4a16_export(self._h, codes.ctypes.data, scales.ctypes.data, _stream(stream)))
        return codes, scales

    def close(self) -> None:
        if self._h is not None and self._h.value:
            lib().svdq_w4a16_destroy(self._h)
        self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class MlpBlock:
    """Y = down(GELU(up(X))) for two prepared NVFP4 layers, with GELU and the
    down layer's quantization fused into the up layer's GEMM epilogue."""

    def __init__(self, up: Layer, down: Layer):
        self.up, self.down = up, down
        self._ws: Optional[torch.Tensor] = None

    def workspace_size(self, M: int) -> int:
        n = ctypes.c_size_t()
        _check(lib().svdq_mlp_workspace_size(self.up._h, self.down._h, M, ctypes.byref(n)))
        return n.value

    def workspace_layout(self, M: int):
        """(codes, scales, T) byte offsets of the down layer's activations in the workspace."""
        off = (ctypes.c_size_t * 3)()
        _check(lib().svdq_mlp_workspace_layout(self.up._h, self.down._h, M, off))
        return tuple(off)

    def workspace(self, M: int) -> torch.Tensor:
        need = self.workspace_size(M)
        if self._ws is None or self._ws.numel() < need:
            self._ws = torch.empty(need, dtype=torch.uint8, device=self.up.device)
        return self._ws

    def forward(self, X: torch.Tensor, out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                stream=None, events=None) -> torch.Tensor:
        self.up._check_io(X, None, workspace)
        M = X.shape[0]
        N = self.down.info().N
        if out is None:
            out = torch.empty(M, N, dtype=torch.bfloat16, device=X.device)
        elif tuple(out.shape) != (M, N) or out.dtype != torch.bfloat16 or not out.is_contiguous():
            raise ValueError(f"out must be a contiguous bfloat16 [{M}, {N}] tensor")
        ws = workspace if workspace is not None else self.workspace(M)
        if events is None:
            _check(lib().svdq_mlp_forward(self.up._h, self.down._h, _ptr(X), M, _ptr(out), _ptr(ws), ws.numel(),
                                          _stream(stream)))
        else:
            arr = (ctypes.c_void_p * 5)(*[e.cuda_event for e in events])
            _check(lib().svdq_mlp_forward_profiled(self.up._h, self.down._h, _ptr(X), M, _ptr(out), _ptr(ws),
                                                   ws.numel(), _stream(stream), arr))
        return out

    __call__ = forward


# ---------------------------------------------------------------- around the quantized layers
_DTYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_ACTIVATION = {None: 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
_NORM = {None: 0, "layer": 1, "rms": 2}
_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


def _place(t: torch.Tensor) -> int:
    """The device of a call's first tensor."""
    device = t.get_device()
    if device < 0:
        raise ValueError("tensors must be CUDA tensors")
    return device


def _operand(name: str, t: torch.Tensor, dtype: torch.dtype, device: int, shape: tuple) -> int:
    """The address of a contiguous tensor of this type, place and shape."""
    if t.dtype is not dtype or t.get_device() != device or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} {list(shape)} tensor on cuda:{device}, "
                         f"got {t.dtype} {list(t.shape)} on {t.device}")
    return t.data_ptr()


def _offsets(name: str, t: torch.Tensor, device: int):
    """The address of the offsets, and of how many sequences they are."""
    n = t.numel()
    if t.dtype is not torch.int32 or t.get_device() != device or t.dim() != 1 or n < 2 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 [sequences + 1] tensor on cuda:{device}")
    return t.data_ptr(), n - 1


def _other_stream(device: int, stream):
    """The torch stream of a call's `stream`, or None where it is the current one."""
    if isinstance(stream, torch.cuda.Stream):
        if stream.device.index != device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{device}")
        return None if stream.cuda_stream == _raw_stream(device) else stream
    handle = _stream(stream)
    if handle == _raw_stream(device):
        return None
    # torch takes handle 0 for none given: an ExternalStream of it would be a stream of torch's pool
    return torch.cuda.ExternalStream(handle, device) if handle else torch.cuda.default_stream(device)


def _on_stream(device: int, other, call, *args, **names):
    """The call with stream `other` as the current one.

    What it makes is allocated there: memory that the caller's stream has freed
    may still be in use on that stream. Results may be used and dropped on the
    caller's stream, and what was given may be dropped after the call."""
    caller = torch.cuda.current_stream(device)
    torch.cuda.set_stream(other)  # of the current device; torch.cuda.stream() takes 6 us more
    try:
        results = call(*args, **names)
    finally:
        torch.cuda.set_stream(caller)
    given = [t for t in (*args, *names.values()) if isinstance(t, torch.Tensor)]
    for t in given:
        t.record_stream(other)
    for t in results if isinstance(results, tuple) else (results,):
        if t is not None and not any(t is g for g in given):
            t.record_stream(caller)
    return results


def _attention_shapes(q, k, v, batch):
    """(dtype, batch, q rows, k rows, q heads, kv heads, dim) of the calls' config, checked."""
    shape, keys = q.shape, k.shape
    if len(shape) != 3 or len(keys) != 3 or keys != v.shape or shape[2] != keys[2]:
        raise ValueError(f"q must be [rows, heads, dim], k and v [rows, heads, dim] alike, got {tuple(shape)}, "
                         f"{tuple(keys)}, {tuple(v.shape)}")
    dtype, device = q.dtype, q.get_device()
    if dtype not in (torch.bfloat16, torch.float16) or k.dtype is not dtype or v.dtype is not dtype:
        raise ValueError("q, k and v must all be bfloat16 or all float16")
    if k.get_device() != device or v.get_device() != device:
        raise ValueError("q, k and v must be on one device")
    return _DTYPE[dtype], batch, shape[0], keys[0], shape[1], keys[1], shape[2]


@functools.lru_cache(maxsize=4096)
def _attention_need(device: int, *shapes: int) -> int:
    """svdq_attention_workspace_size, which goes by the device and the shapes alone."""
    heads, kv_heads, dim = shapes[4:]
    n = ctypes.c_size_t()
    _check(lib().svdq_attention_workspace_size(
        _pack_attention(*shapes, 0, 1.0, heads * dim, dim, kv_heads * dim, dim, kv_heads * dim, dim, *[0] * 8), ctypes.byref(n)))
    return n.value


def attention_workspace_size(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, batch: int = 1) -> int:
    """Bytes of workspace attention() needs for these shapes."""
    device = _place(q)
    with torch.cuda.device(device):
        return _attention_need(device, *_attention_shapes(q, k, v, batch))


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_offsets: Optional[torch.Tensor] = None,
              k_offsets: Optional[torch.Tensor] = None, causal: bool = False, scale: Optional[float] = None,
              out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention of packed sequences (include/svdq.h, svdq_attention_forward).

    q [rows, heads, dim], k and v [rows, kv heads, dim], bfloat16 or float16; views
    are taken as they are (a QKV projection's output need not be split up), as long
    as a head's values are contiguous and the strides multiples of 8. Sequence b
    owns q rows q_offsets[b] to q_offsets[b + 1] and k rows k_offsets[b] to
    k_offsets[b + 1] (int32 on the device; k_offsets defaults to q_offsets, and
    without either all rows are one sequence). causal: the last query of a
    sequence sees every key, the one before it all but one, and so on. scale
    defaults to dim ** -0.5. Rows of `out` that belong to no sequence are not
    written. stream: the call runs on it, behind what is queued there; the
    caller orders it after the work that makes the inputs and before the work
    that uses the result."""
    device = _place(q)
    if device != _current_device():
        with torch.cuda.device(device):
            return attention(q, k, v, q_offsets, k_offsets, causal, scale, out, workspace, stream)
    if stream is not None and (other := _other_stream(device, stream)) is not None:
        return _on_stream(device, other, attention, q, k, v, q_offsets, k_offsets, causal, scale, out, workspace)
    batch, qo, ko = 1, 0, 0
    if q_offsets is not None:
        qo, batch = _offsets("q_offsets", q_offsets, device)
        if k_offsets is None:
            if q.shape[0] != k.shape[0]:
                raise ValueError("k has other rows than q: k_offsets are needed")
            ko = qo
        else:
            ko, k_batch = _offsets("k_offsets", k_offsets, device)
            if k_batch != batch:
                raise ValueError("q_offsets and k_offsets must be of the same length")
    elif k_offsets is not None:
        raise ValueError("k_offsets need q_offsets")
    shapes = _attention_shapes(q, k, v, batch)
    (qr, qh, q1), (kr, kh, k1), (vr, vh, v1) = q.stride(), k.stride(), v.stride()
    if q1 != 1 or k1 != 1 or v1 != 1:
        raise ValueError("the values of a head of q, k and v must be contiguous")
    if out is None:
        out = torch.empty_like(q) if q.is_contiguous() else q.new_empty(tuple(q.shape))
        o = out.data_ptr()
    else:
        o = _operand("out", out, q.dtype, device, q.shape)
    ws, need = 0, _attention_need(device, *shapes)
    if workspace is not None:
        if workspace.dtype is not torch.uint8 or not workspace.is_contiguous() or workspace.get_device() != device:
            raise ValueError("workspace must be a contiguous uint8 tensor on q's device")
        ws, need = workspace.data_ptr(), workspace.numel()
    elif need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        ws = workspace.data_ptr()
    args = _pack_attention(*shapes, 1 if causal else 0, shapes[6] ** -0.5 if scale is None else scale, qr, qh, kr, kh, vr, vh,
                           q.data_ptr(), k.data_ptr(), v.data_ptr(), qo, ko, o, ws, need)
    _check(lib().svdq_attention_forward(args, _raw_stream(device)))
    return out


def linear(X: torch.Tensor, W: torch.Tensor, bias: Optional[torch.Tensor] = None, activation: Optional[str] = None,
           residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """residual + activation(X W + bias) for a layer whose weight stays in 16 bits
    (include/svdq.h, svdq_dense_linear_forward): X [M, K], W [K, N], bias [N],
    residual and out [M, N], all bfloat16 or all float16; activation None, "relu",
    "silu", "gelu" or "gelu_tanh". out may be the residual. stream as in attention()."""
    dtype = X.dtype
    if X.dim() != 2 or W.dim() != 2 or dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("X and W must be bfloat16 or float16 matrices")
    act = _ACTIVATION.get(activation)
    if act is None:
        raise ValueError(f"unknown activation {activation!r}")
    device = _place(X)
    if device != _current_device():
        with torch.cuda.device(device):
            return linear(X, W, bias, activation, residual, out, stream)
    if stream is not None and (other := _other_stream(device, stream)) is not None:
        return _on_stream(device, other, linear, X, W, bias, activation, residual, out)
    (M, K), N = X.shape, W.shape[1]
    if not X.is_contiguous():
        raise ValueError("X must be contiguous")
    w = _operand("W", W, dtype, device, (K, N))
    b = 0 if bias is None else _operand("bias", bias, dtype, device, (N,))
    r = 0 if residual is None else _operand("residual", residual, dtype, device, (M, N))
    if out is None:
        out = X.new_empty((M, N)) if residual is None else torch.empty_like(residual)
        y = out.data_ptr()
    else:
        y = _operand("out", out, dtype, device, (M, N))
    args = _pack_dense_linear(_DTYPE[dtype], act, M, K, N, X.data_ptr(), w, b, r, y)
    _check(lib().svdq_dense_linear_forward(args, _raw_stream(device)))
    return out


def residual_norm(x: torch.Tensor, y: Optional[torch.Tensor] = None, *, offsets: Optional[torch.Tensor] = None,
                  gate: Optional[torch.Tensor] = None, residual_scale: float = 1.0, post_norm: Optional[str] = None,
                  post_weight: Optional[torch.Tensor] = None, post_bias: Optional[torch.Tensor] = None,
                  norm: Optional[str] = "rms", weight: Optional[torch.Tensor] = None,
                  bias: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                  shift: Optional[torch.Tensor] = None, eps: float = 1e-6, dtype: Optional[torch.dtype] = None,
                  out_x: Optional[torch.Tensor] = None, out_h: Optional[torch.Tensor] = None, stream=None):
    """The norms after and before a block with the block's gate and residual
    (include/svdq.h, svdq_residual_norm); returns (x', h):

        x' = residual_scale x + gate * post_norm(y)
        h  = norm(x') * (1 + scale) + shift

    x [rows, dim] is the residual stream (float32, or the type of y), y the
    block's output. Norms are "layer", "rms" or None, with weights and biases of
    [dim]. gate, scale and shift are [sequences, dim], row b for the tokens
    offsets[b] to offsets[b + 1] (without offsets, one row for all). Without y
    (the first norm of a model) x' is x itself and only h is computed, in `dtype`
    (that of x where x is not float32); with norm None h is None. out_x may be x,
    out_h may be y. Rows that belong to no sequence are not written. stream as in
    attention()."""
    x_kind = x.dtype
    if x.dim() != 2 or x_kind not in _DTYPE:
        raise ValueError("x must be a [rows, dim] tensor of bfloat16, float16 or float32")
    if norm not in _NORM or post_norm not in _NORM:
        raise ValueError(f"unknown norm {norm if norm not in _NORM else post_norm!r}")
    kind = y.dtype if y is not None else dtype if dtype is not None else x_kind
    if (kind is not torch.bfloat16 and kind is not torch.float16) or (x_kind is not kind and x_kind is not torch.float32):
        raise ValueError("y and h must be bfloat16 or float16, x of the same type or float32")
    if dtype is not None and dtype != kind:
        raise ValueError("dtype must be that of y")
    device = _place(x)
    if device != _current_device():
        with torch.cuda.device(device):
            return residual_norm(x, y, offsets=offsets, gate=gate, residual_scale=residual_scale, post_norm=post_norm,
                                 post_weight=post_weight, post_bias=post_bias, norm=norm, weight=weight, bias=bias,
                                 scale=scale, shift=shift, eps=eps, dtype=dtype, out_x=out_x, out_h=out_h, stream=stream)
    if stream is not None and (other := _other_stream(device, stream)) is not None:
        return _on_stream(device, other, residual_norm, x, y, offsets=offsets, gate=gate, residual_scale=residual_scale,
                          post_norm=post_norm, post_weight=post_weight, post_bias=post_bias, norm=norm, weight=weight,
                          bias=bias, scale=scale, shift=shift, eps=eps, dtype=dtype, out_x=out_x, out_h=out_h)
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    shape = x.shape
    rows, dim = shape
    seqs, off, x_out, h_out = 1, None, 0, 0
    if offsets is not None:
        off, seqs = _offsets("offsets", offsets, device)
    of_row, of_seq = (dim,), (seqs, dim)
    if seqs == 1:  # one row for all may come without its first dimension
        gate, scale, shift = (None if t is None else t.view(1, -1) if t.dim() == 1 else t for t in (gate, scale, shift))
    if y is not None:
        if out_x is None:
            out_x = torch.empty_like(x)
            x_out = out_x.data_ptr()
        else:
            x_out = _operand("out_x", out_x, x_kind, device, shape)
    elif out_x is not None:
        raise ValueError("without y there is no out_x")
    if norm is not None:
        if out_h is None:
            out_h = torch.empty_like(x, dtype=kind) if y is None else torch.empty_like(y)
            h_out = out_h.data_ptr()
        else:
            h_out = _operand("out_h", out_h, kind, device, shape)
    elif out_h is not None:
        raise ValueError("without a norm there is no out_h")
    args = _pack_residual_norm(
        _DTYPE[kind], _DTYPE[x_kind], rows, dim, seqs, _NORM[post_norm], _NORM[norm], residual_scale, eps,
        x.data_ptr(), 0 if y is None else _operand("y", y, kind, device, shape), x_out, h_out,
        0 if gate is None else _operand("gate", gate, kind, device, of_seq),
        0 if post_weight is None else _operand("post_weight", post_weight, kind, device, of_row),
        0 if post_bias is None else _operand("post_bias", post_bias, kind, device, of_row),
        0 if weight is None else _operand("weight", weight, kind, device, of_row),
        0 if bias is None else _operand("bias", bias, kind, device, of_row),
        0 if scale is None else _operand("scale", scale, kind, device, of_seq),
        0 if shift is None else _operand("shift", shift, kind, device, of_seq), off or 0)
    _check(lib().svdq_residual_norm(args, _raw_stream(device)))
    return x if y is None else out_x, out_h


def selftest_operator_wait(kernels: int, stream=None) -> None:
    """A wait in vain that operator_status() then reports (include/svdq.h, svdq_selftest_operator_wait)."""
    _check(lib().svdq_selftest_operator_wait(kernels, _stream(stream)))


def operator_status(stream=None) -> Status:
    """Reads and clears the current device's status word of attention and linear."""
    return Status(lib().svdq_operator_status(_stream(stream)))
