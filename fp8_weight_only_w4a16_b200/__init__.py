"""B200-native weight-only skinny GEMM: y[M,N] = x[M,K] . W^T, M = 1..16,
with W kept in HBM as NVFP4 (E2M1 codes + UE4M3 per-16 scales + FP32 global)
or FP8 E4M3 (+ FP32 per output channel), FP16 activations, FP32 accumulation;
products for any number of tokens, grouped by expert (the same formats) or in
8-bit integers; and the verification of drafted tokens.

This module is a thin binding over ``libskinny.so`` (whose C ABI is
``include/skinny.h``): it turns numpy arrays and torch tensors into pointers,
sizes and a stream handle, calls the library (by ctypes, or from ``_binding.so``
where a call is short), and raises ``SkinnyError`` on a non-zero status.  Every
step of the GEMM runs in the library's CUDA kernels;
there is no fallback: if the library is missing, the first call raises.
"""
from __future__ import annotations

import ctypes
import dataclasses
import os
import threading

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIBRARY_PATH = os.path.join(_PKG, "libskinny.so")

OK = 0
ERR_INVALID_ARG = -1
ERR_UNSUPPORTED = -2
ERR_ALIGNMENT = -3
ERR_CUDA = -4
ERR_WORKSPACE = -5

OUT_F16 = 0
OUT_F32 = 1
FMT_NVFP4 = 0
FMT_FP8 = 1
MAX_M = 16
MAX_GROUP = 8
MAX_EXPERTS = 512
PROB_F16 = 0
PROB_F32 = 1
PROB_BF16 = 2

_lock = threading.Lock()
_lib = None


class GroupMember(ctypes.Structure):
    """skinny_nvfp4_group_member of include/skinny.h."""
    _fields_ = [("x", ctypes.c_void_p), ("w_packed", ctypes.c_void_p), ("global_scale", ctypes.c_float),
                ("N", ctypes.c_int64), ("y", ctypes.c_void_p)]


class SkinnyError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__("%s: %s (%d)" % (what, status_string(status), status))


def library() -> ctypes.CDLL:
    """Load libskinny.so (built by ``__graft_entry__.build()``); raise if absent."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIBRARY_PATH):
                raise RuntimeError("libskinny.so is not built (%s); run __graft_entry__.build()" % LIBRARY_PATH)
            lib = ctypes.CDLL(LIBRARY_PATH)
            p, i64, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
            sigs = {
                "skinny_status_string": (ctypes.c_char_p, [ctypes.c_int]),
                "skinny_version": (ctypes.c_int, []),
                "skinny_nvfp4_packed_bytes": (sz, [i64, i64]),
                "skinny_pack_nvfp4": (ctypes.c_int, [p, p, i64, i64, p]),
                "skinny_unpack_nvfp4": (ctypes.c_int, [p, i64, i64, p, p]),
                "skinny_fp8_packed_bytes": (sz, [i64, i64]),
                "skinny_pack_fp8": (ctypes.c_int, [p, i64, i64, p]),
                "skinny_unpack_fp8": (ctypes.c_int, [p, i64, i64, p]),
                "skinny_workspace_bytes": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, i64, i64, ctypes.POINTER(sz)]),
                "skinny_nvfp4_gemm": (ctypes.c_int, [p, ctypes.c_int, i64, p, ctypes.c_float, i64, p, ctypes.c_int,
                                                     p, sz, p]),
                "skinny_fp8_gemm": (ctypes.c_int, [p, ctypes.c_int, i64, p, p, i64, p, ctypes.c_int, p, sz, p]),
                "skinny_device_error": (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(ctypes.c_uint)]),
                "skinny_nvfp4_gemm_static_ws": (ctypes.c_int, [p, ctypes.c_int, i64, p, ctypes.c_float, i64, p,
                                                               ctypes.c_int, p]),
                "skinny_nvfp4_gemm_argmax": (ctypes.c_int, [p, ctypes.c_int, i64, p, ctypes.c_float, i64, p, p, p,
                                                            sz, p]),
                "skinny_pack_nvfp4_gate_up": (ctypes.c_int, [p, p, i64, i64, p]),
                "skinny_debug_schedule": (ctypes.c_int, [i64, i64, ctypes.c_int, ctypes.c_int, p, ctypes.c_int,
                                                         ctypes.POINTER(ctypes.c_int)]),
                "skinny_nvfp4_gemm_add": (ctypes.c_int, [p, ctypes.c_int, i64, p, ctypes.c_float, i64, p, p,
                                                         ctypes.c_int, p, sz, p]),
                "skinny_fp8_gemm_add": (ctypes.c_int, [p, ctypes.c_int, i64, p, p, i64, p, p, ctypes.c_int, p, sz,
                                                       p]),
                "skinny_nvfp4_gemm_silu_mul": (ctypes.c_int, [p, ctypes.c_int, i64, p, ctypes.c_float, i64, p,
                                                              ctypes.c_int, p, sz, p]),
                "skinny_static_workspace_capacity": (sz, []),
                "skinny_stream_read": (ctypes.c_int, [p, sz, ctypes.c_int, p, p]),
                "skinny_nvfp4_gemm_grouped": (ctypes.c_int, [ctypes.POINTER(GroupMember), ctypes.c_int,
                                                             ctypes.c_int, i64, ctypes.c_int, p, sz, p]),
                "skinny_tile_workspace_bytes": (ctypes.c_int, [ctypes.POINTER(sz)]),
                "skinny_experts_packed_bytes": (sz, [ctypes.c_int, i64, i64, i64, ctypes.c_int]),
                "skinny_pack_experts": (ctypes.c_int, [ctypes.c_int, p, p, i64, i64, i64, ctypes.c_int, p, p]),
                "skinny_gemm_experts": (ctypes.c_int, [ctypes.c_int, p, i64, i64, p, i64, p, p, i64, p, ctypes.c_int,
                                                       p, sz, p]),
                "skinny_gemm_experts_silu_mul": (ctypes.c_int, [ctypes.c_int, p, i64, i64, p, i64, p, p, i64, p,
                                                                ctypes.c_int, p, sz, p]),
                "skinny_quantize_int8": (ctypes.c_int, [p, ctypes.c_int, i64, i64, p, p, p]),
                "skinny_int8_gemm": (ctypes.c_int, [p, p, i64, i64, p, p, i64, p, ctypes.c_int, p, sz, p]),
                "skinny_tile_device_error": (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(ctypes.c_uint)]),
                "skinny_debug_tile_width": (ctypes.c_int, [ctypes.c_int, i64, i64, i64, i64, ctypes.c_int, ctypes.c_int,
                                                           ctypes.c_int, p]),
                "skinny_debug_tile_rings": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, p]),
                "skinny_debug_tile_columns": (ctypes.c_int, [ctypes.c_int, ctypes.c_int]),
                "skinny_verify_draft": (ctypes.c_int, [p, i64, i64, p, i64, i64, ctypes.c_int, p, p, p, i64, i64, i64,
                                                       p, p, p]),
                "skinny_debug_static_workspace_address": (ctypes.c_int, [ctypes.POINTER(ctypes.c_void_p)]),
            }
            for name, (res, args) in sigs.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
    return _lib


def status_string(status: int) -> str:
    return library().skinny_status_string(int(status)).decode()


def _check(status: int, what: str):
    if status != OK:
        raise SkinnyError(status, what)


def _np_ptr(a: np.ndarray) -> int:
    return a.ctypes.data


# ---------------------------------------------------------------------------
# Host-side packing
# ---------------------------------------------------------------------------

def nvfp4_packed_bytes(N: int, K: int) -> int:
    """Bytes of the packed NVFP4 layout (codes and block scales)."""
    return int(library().skinny_nvfp4_packed_bytes(int(N), int(K)))


def fp8_packed_bytes(N: int, K: int) -> int:
    return int(library().skinny_fp8_packed_bytes(int(N), int(K)))


def pack_nvfp4(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """Logical codes [N, K/2] (low nibble = even k) and UE4M3 scales [N, K/16] ->
    the packed uint8 buffer (tiles of codes with their block scales)."""
    codes = np.ascontiguousarray(codes, dtype=np.uint8)
    scales = np.ascontiguousarray(scales, dtype=np.uint8)
    N, K = codes.shape[0], codes.shape[1] * 2
    if scales.shape != (N, K // 16):
        raise ValueError("scales must be [N, K/16]")
    nb = nvfp4_packed_bytes(N, K)
    if nb == 0:
        raise SkinnyError(ERR_INVALID_ARG, "pack_nvfp4 shape")
    out = np.empty(nb, np.uint8)
    _check(library().skinny_pack_nvfp4(_np_ptr(codes), _np_ptr(scales), N, K, _np_ptr(out)), "skinny_pack_nvfp4")
    return out


def unpack_nvfp4(packed: np.ndarray, N: int, K: int):
    packed = np.ascontiguousarray(packed, dtype=np.uint8)
    codes, scales = np.empty((N, K // 2), np.uint8), np.empty((N, K // 16), np.uint8)
    _check(library().skinny_unpack_nvfp4(_np_ptr(packed), N, K, _np_ptr(codes), _np_ptr(scales)),
           "skinny_unpack_nvfp4")
    return codes, scales


def pack_fp8(q: np.ndarray) -> np.ndarray:
    q = np.ascontiguousarray(q, dtype=np.uint8)
    N, K = q.shape
    nb = fp8_packed_bytes(N, K)
    if nb == 0:
        raise SkinnyError(ERR_INVALID_ARG, "pack_fp8 shape")
    out = np.empty(nb, np.uint8)
    _check(library().skinny_pack_fp8(_np_ptr(q), N, K, _np_ptr(out)), "skinny_pack_fp8")
    return out


def unpack_fp8(packed: np.ndarray, N: int, K: int) -> np.ndarray:
    packed = np.ascontiguousarray(packed, dtype=np.uint8)
    q = np.empty((N, K), np.uint8)
    _check(library().skinny_unpack_fp8(_np_ptr(packed), N, K, _np_ptr(q)), "skinny_unpack_fp8")
    return q


# ---------------------------------------------------------------------------
# Device GEMMs (torch supplies device memory and the stream)
#
# With `stream`, a call runs on that stream, and the outputs that it allocates
# belong to it, as under torch.cuda.stream(stream).
# ---------------------------------------------------------------------------

@dataclasses.dataclass
class PackedNVFP4:
    data: "object"           # torch.uint8 device tensor (packed tiles: codes + block scales)
    global_scale: float
    N: int
    K: int

    @classmethod
    def from_logical(cls, codes: np.ndarray, scales: np.ndarray, global_scale: float, device="cuda"):
        import torch

        return cls(torch.from_numpy(pack_nvfp4(codes, scales)).to(device), float(global_scale), codes.shape[0],
                   codes.shape[1] * 2)

    @property
    def fmt(self) -> int:
        return FMT_NVFP4

    @property
    def nbytes(self) -> int:
        return int(self.data.numel())


@dataclasses.dataclass
class PackedFP8:
    codes: "object"          # torch.uint8 device tensor (packed layout)
    channel_scale: "object"  # torch.float32 device tensor [N]
    N: int
    K: int

    @classmethod
    def from_logical(cls, q: np.ndarray, channel_scale: np.ndarray, device="cuda"):
        import torch

        return cls(torch.from_numpy(pack_fp8(q)).to(device),
                   torch.from_numpy(np.ascontiguousarray(channel_scale, np.float32)).to(device), q.shape[0], q.shape[1])

    @property
    def fmt(self) -> int:
        return FMT_FP8

    @property
    def nbytes(self) -> int:
        return int(self.codes.numel() + 4 * self.channel_scale.numel())


def workspace_bytes(fmt: int, M: int, N: int, K: int) -> int:
    """Split-K workspace size for one GEMM on the current device."""
    b = ctypes.c_size_t(0)
    _check(library().skinny_workspace_bytes(int(fmt), int(M), int(N), int(K), ctypes.byref(b)),
           "skinny_workspace_bytes")
    return int(b.value)


def make_workspace(fmt: int, M: int, N: int, K: int, device="cuda"):
    """A zero-filled workspace (its partial-sum slots must start at zero)."""
    import torch

    return torch.zeros(workspace_bytes(fmt, M, N, K), dtype=torch.uint8, device=device)


def _stream_handle(stream) -> int:
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


def _empty(shape, dtype, device, stream):
    """An output of a call on `stream`, in that stream's memory: a block of the current stream's
    may still be read by what is pending there."""
    import torch

    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def gemm_into(y, x, w, workspace=None, stream=None) -> None:
    """y[M, N] = x[M, K] . W^T on the device (y float16 or float32, preallocated)."""
    import torch

    M, K = x.shape
    if x.dtype != torch.float16 or not x.is_contiguous() or K != w.K:
        raise ValueError("x must be a contiguous float16 [M, %d] tensor" % w.K)
    if y.shape != (M, w.N) or not y.is_contiguous() or y.dtype not in (torch.float16, torch.float32):
        raise ValueError("y must be a contiguous float16/float32 [M, N] tensor")
    out = OUT_F32 if y.dtype == torch.float32 else OUT_F16
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    h = _stream_handle(stream)
    lib = library()
    if w.fmt == FMT_NVFP4:
        st = lib.skinny_nvfp4_gemm(x.data_ptr(), M, K, w.data.data_ptr(), ctypes.c_float(w.global_scale), w.N,
                                   y.data_ptr(), out, ws_ptr, ws_bytes, h)
        _check(st, "skinny_nvfp4_gemm")
    else:
        st = lib.skinny_fp8_gemm(x.data_ptr(), M, K, w.codes.data_ptr(), w.channel_scale.data_ptr(), w.N,
                                 y.data_ptr(), out, ws_ptr, ws_bytes, h)
        _check(st, "skinny_fp8_gemm")


def gemm_add_into(y, x, w, residual, workspace=None, stream=None) -> None:
    """y[M, N] = x . W^T + residual, the add in FP32 before the one output
    rounding; residual has y's shape and dtype and may be y itself."""
    import torch

    M, K = x.shape
    if x.dtype != torch.float16 or not x.is_contiguous() or K != w.K:
        raise ValueError("x must be a contiguous float16 [M, %d] tensor" % w.K)
    if y.shape != (M, w.N) or not y.is_contiguous() or y.dtype not in (torch.float16, torch.float32):
        raise ValueError("y must be a contiguous float16/float32 [M, N] tensor")
    if residual.shape != y.shape or residual.dtype != y.dtype or not residual.is_contiguous():
        raise ValueError("residual must be a contiguous tensor of y's shape and dtype")
    out = OUT_F32 if y.dtype == torch.float32 else OUT_F16
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    h = _stream_handle(stream)
    lib = library()
    if w.fmt == FMT_NVFP4:
        st = lib.skinny_nvfp4_gemm_add(x.data_ptr(), M, K, w.data.data_ptr(), ctypes.c_float(w.global_scale), w.N,
                                       residual.data_ptr(), y.data_ptr(), out, ws_ptr, ws_bytes, h)
        _check(st, "skinny_nvfp4_gemm_add")
    else:
        st = lib.skinny_fp8_gemm_add(x.data_ptr(), M, K, w.codes.data_ptr(), w.channel_scale.data_ptr(), w.N,
                                     residual.data_ptr(), y.data_ptr(), out, ws_ptr, ws_bytes, h)
        _check(st, "skinny_fp8_gemm_add")


def gemm_grouped_into(ys, xs, ws, workspace=None, stream=None) -> None:
    """ys[i][M, N_i] = xs[i][M, K] . W_i^T for every i, in ONE launch (NVFP4
    weights of the same K; ys all float16 or all float32, preallocated)."""
    import torch

    if not (len(ys) == len(xs) == len(ws)) or not 1 <= len(ws) <= MAX_GROUP:
        raise ValueError("ys, xs and ws must have the same length, 1..%d" % MAX_GROUP)
    M, K = xs[0].shape
    dt = ys[0].dtype
    members = (GroupMember * len(ws))()
    for i, (y, x, w) in enumerate(zip(ys, xs, ws)):
        if w.fmt != FMT_NVFP4 or w.K != K:
            raise ValueError("grouped GEMMs take NVFP4 weights of one K")
        if x.dtype != torch.float16 or not x.is_contiguous() or x.shape != (M, K):
            raise ValueError("every x must be a contiguous float16 [%d, %d] tensor" % (M, K))
        if y.shape != (M, w.N) or not y.is_contiguous() or y.dtype != dt or dt not in (torch.float16, torch.float32):
            raise ValueError("every y must be a contiguous [M, N_i] tensor of one dtype (float16 or float32)")
        members[i] = GroupMember(x.data_ptr(), w.data.data_ptr(), w.global_scale, w.N, y.data_ptr())
    out = OUT_F32 if dt == torch.float32 else OUT_F16
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = library().skinny_nvfp4_gemm_grouped(members, len(ws), M, K, out, ws_ptr, ws_bytes, _stream_handle(stream))
    _check(st, "skinny_nvfp4_gemm_grouped")


def gemm(x, w, out_dtype=None, workspace=None, stream=None):
    """Allocate y and compute y = x . W^T (float16 output unless out_dtype says otherwise)."""
    import torch

    y = _empty((x.shape[0], w.N), out_dtype or torch.float16, x.device, stream)
    gemm_into(y, x, w, workspace=workspace, stream=stream)
    return y


def pack_nvfp4_gate_up(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """Pack gate+up weights (rows 0..F-1 gate, F..2F-1 up) for the fused SiLU*mul GEMM."""
    codes = np.ascontiguousarray(codes, dtype=np.uint8)
    scales = np.ascontiguousarray(scales, dtype=np.uint8)
    n2, half_k = codes.shape
    K = 2 * half_k
    if n2 % 2 or scales.shape != (n2, K // 16):
        raise ValueError("codes [2F, K/2] and scales [2F, K/16] expected")
    out = np.zeros(nvfp4_packed_bytes(n2, K), np.uint8)
    _check(library().skinny_pack_nvfp4_gate_up(codes.ctypes.data, scales.ctypes.data, n2 // 2, K, out.ctypes.data),
           "skinny_pack_nvfp4_gate_up")
    return out


@dataclasses.dataclass
class PackedGateUp:
    """Gate+up NVFP4 weights packed for gemm_silu_mul: F outputs, 2F weight rows."""
    data: "object"
    global_scale: float
    F: int
    K: int

    @classmethod
    def from_logical(cls, codes: np.ndarray, scales: np.ndarray, global_scale: float, device="cuda"):
        import torch

        return cls(torch.from_numpy(pack_nvfp4_gate_up(codes, scales)).to(device), float(global_scale),
                   codes.shape[0] // 2, codes.shape[1] * 2)

    @property
    def fmt(self) -> int:
        return FMT_NVFP4

    @property
    def N(self) -> int:
        """Weight rows (gate and up): the GEMM's N, e.g. for workspace_bytes."""
        return 2 * self.F


def gemm_silu_mul_into(y, x, w: "PackedGateUp", workspace=None, stream=None) -> None:
    """y[M, F] = silu(x . Wgate^T) * (x . Wup^T) (y float16 or float32, preallocated)."""
    import torch

    if not isinstance(w, PackedGateUp):
        raise TypeError("gemm_silu_mul takes weights packed by PackedGateUp / pack_nvfp4_gate_up")
    M, K = x.shape
    if x.dtype != torch.float16 or not x.is_contiguous() or K != w.K:
        raise ValueError("x must be a contiguous float16 [M, %d] tensor" % w.K)
    if y.shape != (M, w.F) or not y.is_contiguous() or y.dtype not in (torch.float16, torch.float32):
        raise ValueError("y must be a contiguous float16/float32 [M, F] tensor")
    out = OUT_F32 if y.dtype == torch.float32 else OUT_F16
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = library().skinny_nvfp4_gemm_silu_mul(x.data_ptr(), M, K, w.data.data_ptr(), ctypes.c_float(w.global_scale),
                                              w.F, y.data_ptr(), out, ws_ptr, ws_bytes, _stream_handle(stream))
    _check(st, "skinny_nvfp4_gemm_silu_mul")


def gemm_silu_mul(x, w: "PackedGateUp", out_dtype=None, workspace=None, stream=None):
    """Allocate y [M, F] and compute the fused gate+up GEMM with SiLU*mul."""
    import torch

    y = _empty((x.shape[0], w.F), out_dtype or torch.float16, x.device, stream)
    gemm_silu_mul_into(y, x, w, workspace=workspace, stream=stream)
    return y


def gemm_argmax_into(idx, val, x, w, workspace, stream=None) -> None:
    """Per token m: idx[m] = argmax_n y[m, n], val[m] = y[m, idx[m]] for y = x . W^T
    (NVFP4 W), without writing y.  idx int32 [M], val float32 [M]; the workspace
    (zero-filled, from make_workspace) is required."""
    import torch

    M, K = x.shape
    if x.dtype != torch.float16 or not x.is_contiguous() or K != w.K:
        raise ValueError("x must be a contiguous float16 [M, %d] tensor" % w.K)
    if w.fmt != FMT_NVFP4:
        raise ValueError("the fused argmax takes NVFP4 weights")
    if idx.shape != (M,) or idx.dtype != torch.int32 or val.shape != (M,) or val.dtype != torch.float32:
        raise ValueError("idx must be int32 [M] and val float32 [M]")
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = library().skinny_nvfp4_gemm_argmax(x.data_ptr(), M, K, w.data.data_ptr(), ctypes.c_float(w.global_scale),
                                            w.N, idx.data_ptr(), val.data_ptr(), ws_ptr, ws_bytes,
                                            _stream_handle(stream))
    _check(st, "skinny_nvfp4_gemm_argmax")


def gemm_argmax(x, w, workspace, stream=None):
    """Allocate and return (idx int32 [M], val float32 [M]): see gemm_argmax_into."""
    import torch

    idx = _empty((x.shape[0],), torch.int32, x.device, stream)
    val = _empty((x.shape[0],), torch.float32, x.device, stream)
    gemm_argmax_into(idx, val, x, w, workspace, stream=stream)
    return idx, val


def device_error(clear: bool = True) -> int:
    """Synchronise and read the device-side error word (0 = no wait gave up)."""
    v = ctypes.c_uint(0)
    _check(library().skinny_device_error(1 if clear else 0, ctypes.byref(v)), "skinny_device_error")
    return int(v.value)


# ---------------------------------------------------------------------------
# Products for any number of tokens: experts and 8-bit integers
#
# With `stream`, a call runs on that stream, and the outputs that it allocates
# belong to it, as under torch.cuda.stream(stream).
# ---------------------------------------------------------------------------

_native = None


def binding():
    """The compiled binding of the calls below (``_binding.so``, built by
    ``__graft_entry__.build()``), given the loaded library's functions; raise if absent."""
    global _native
    if _native is None:
        import importlib.util

        import torch  # noqa: F401  (its libraries are loaded first)

        path = os.path.join(_PKG, "_binding.so")
        if not os.path.exists(path):
            raise RuntimeError("_binding.so is not built (%s); run __graft_entry__.build()" % path)
        spec = importlib.util.spec_from_file_location(__name__ + "._binding", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        lib = library()
        module.bind(SkinnyError, *(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in (
            "skinny_gemm_experts", "skinny_gemm_experts_silu_mul", "skinny_quantize_int8", "skinny_int8_gemm",
            "skinny_verify_draft", "skinny_experts_packed_bytes")))
        _native = module
    return _native


def _given(*outputs):
    if any(t is None for t in outputs):
        raise ValueError("the output tensors must be given")


def tile_workspace_bytes() -> int:
    """Size of the experts' and int8 products' workspace on the current device."""
    b = ctypes.c_size_t(0)
    _check(library().skinny_tile_workspace_bytes(ctypes.byref(b)), "skinny_tile_workspace_bytes")
    return int(b.value)


def make_experts_workspace(device="cuda"):
    """A zero-filled workspace for gemm_experts and gemm_experts_silu_mul; it
    serves calls of any shape in turn, but not two that can run at the same time."""
    import torch

    with torch.cuda.device(device):
        return torch.zeros(tile_workspace_bytes(), dtype=torch.uint8, device=device)


def make_int8_workspace(device="cuda"):
    """A zero-filled workspace for gemm_int8 (alike, and interchangeable with, make_experts_workspace's)."""
    return make_experts_workspace(device)


def _pack_experts(fmt, codes, scales, E, N, K, gate_up):
    import torch

    nb = int(library().skinny_experts_packed_bytes(fmt, E, N, K, int(gate_up)))
    if nb == 0:
        raise SkinnyError(ERR_INVALID_ARG, "pack_experts shape")
    out = torch.empty(nb, dtype=torch.uint8, device=codes.device)
    with torch.cuda.device(codes.device):
        st = library().skinny_pack_experts(fmt, codes.data_ptr(), scales.data_ptr() if scales is not None else None,
                                           E, N, K, int(gate_up), out.data_ptr(), _stream_handle(None))
    _check(st, "skinny_pack_experts")
    return out


def _device_tensor(a, dtype, device):
    import torch

    t = a if isinstance(a, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(a))
    if t.dtype != dtype:
        raise ValueError("a %s tensor expected, got %s" % (dtype, t.dtype))
    return t.to(device).contiguous()


@dataclasses.dataclass
class PackedExpertsNVFP4:
    """E experts of N x K NVFP4 weights, packed for gemm_experts or (gate_up:
    rows 0..N/2-1 gate, N/2..N-1 up) for gemm_experts_silu_mul."""
    data: "object"           # torch.uint8 device tensor
    scale: "object"          # torch.float32 device tensor [E]: one scale per expert
    E: int
    N: int
    K: int
    gate_up: bool

    @classmethod
    def from_logical(cls, codes, scales, expert_scale, gate_up=False, device="cuda"):
        """codes [E, N, K/2] uint8 (low nibble = even k), scales [E, N, K/16]
        UE4M3 bytes, expert_scale [E] float32; numpy arrays or torch tensors."""
        import torch

        codes, scales = (_device_tensor(a, torch.uint8, device) for a in (codes, scales))
        expert_scale = _device_tensor(expert_scale, torch.float32, device)
        if codes.dim() != 3:
            raise ValueError("codes must be [E, N, K/2]")
        E, N, K = codes.shape[0], codes.shape[1], codes.shape[2] * 2
        if tuple(scales.shape) != (E, N, K // 16) or tuple(expert_scale.shape) != (E,):
            raise ValueError("scales must be [E, N, K/16] and expert_scale [E]")
        if bool((scales >= 0x7F).any()):
            raise ValueError("block scales must be finite non-negative UE4M3 bytes")
        return cls(_pack_experts(FMT_NVFP4, codes, scales, E, N, K, gate_up), expert_scale, E, N, K, bool(gate_up))

    @property
    def fmt(self) -> int:
        return FMT_NVFP4


@dataclasses.dataclass
class PackedExpertsFP8:
    """E experts of N x K FP8 E4M3 weights with a scale per expert and output
    channel, packed as PackedExpertsNVFP4."""
    data: "object"           # torch.uint8 device tensor
    scale: "object"          # torch.float32 device tensor [E, N]
    E: int
    N: int
    K: int
    gate_up: bool

    @classmethod
    def from_logical(cls, q, channel_scale, gate_up=False, device="cuda"):
        """q [E, N, K] E4M3 bytes (uint8), channel_scale [E, N] float32."""
        import torch

        q = _device_tensor(q, torch.uint8, device)
        channel_scale = _device_tensor(channel_scale, torch.float32, device)
        if q.dim() != 3 or tuple(channel_scale.shape) != tuple(q.shape[:2]):
            raise ValueError("q must be [E, N, K] and channel_scale [E, N]")
        if bool(((q & 0x7F) == 0x7F).any()):
            raise ValueError("E4M3 codes must not be NaN")
        E, N, K = q.shape
        return cls(_pack_experts(FMT_FP8, q, None, E, N, K, gate_up), channel_scale, E, N, K, bool(gate_up))

    @property
    def fmt(self) -> int:
        return FMT_FP8


def _gemm_experts(y, x, w, offsets, out_dtype, workspace, stream, silu):
    """The experts' product into y, or into a new tensor of out_dtype; returns it."""
    if w.gate_up != silu:
        raise TypeError("gemm_experts takes experts packed without gate_up, gemm_experts_silu_mul with it")
    return (_native or binding()).gemm_experts(silu, y, x, w.fmt, w.E, w.N, w.K, w.data, w.scale, offsets, out_dtype,
                                               workspace, stream)


def gemm_experts_into(y, x, w, offsets, workspace=None, stream=None) -> None:
    """y[r, N] = x[r, K] . W_e^T for the rows offsets[e] <= r < offsets[e+1] of
    every expert e.  x float16 [T, K], sorted by expert; offsets int32 [E+1] on
    the device; y float16 or float32, preallocated: rows of no expert are left
    as they are.  T may be any number."""
    _given(y)
    _gemm_experts(y, x, w, offsets, None, workspace, stream, False)


def gemm_experts(x, w, offsets, out_dtype=None, workspace=None, stream=None):
    """Allocate y [T, N] (float16 unless out_dtype says otherwise): see
    gemm_experts_into.  Rows of no expert are not written."""
    return _gemm_experts(None, x, w, offsets, out_dtype, workspace, stream, False)


def gemm_experts_silu_mul_into(y, x, w, offsets, workspace=None, stream=None) -> None:
    """y[r, N/2] = silu(gate) * up of the rows' experts (packed with gate_up):
    otherwise as gemm_experts_into."""
    _given(y)
    _gemm_experts(y, x, w, offsets, None, workspace, stream, True)


def gemm_experts_silu_mul(x, w, offsets, out_dtype=None, workspace=None, stream=None):
    """Allocate y [T, N/2]: see gemm_experts_silu_mul_into."""
    return _gemm_experts(None, x, w, offsets, out_dtype, workspace, stream, True)


@dataclasses.dataclass
class WeightInt8:
    """N x K 8-bit integer weights, as they are, with one scale per output channel."""
    codes: "object"          # torch.int8 device tensor [N, K]
    channel_scale: "object"  # torch.float32 device tensor [N]

    def __post_init__(self):
        import torch

        if self.codes.dim() != 2 or self.codes.dtype != torch.int8 or not self.codes.is_contiguous():
            raise ValueError("codes must be a contiguous int8 [N, K] tensor")
        s = self.channel_scale
        if tuple(s.shape) != (self.codes.shape[0],) or s.dtype != torch.float32 or not s.is_contiguous():
            raise ValueError("channel_scale must be a contiguous float32 [N] tensor")

    @property
    def N(self) -> int:
        return int(self.codes.shape[0])

    @property
    def K(self) -> int:
        return int(self.codes.shape[1])


def quantize_int8_into(q, row_scale, x, stream=None) -> None:
    """Rows of x (float16 or float32 [M, K]) to 8-bit integers: row_scale =
    max|x| / 127, q = round(x / row_scale).  q int8 [M, K], row_scale float32 [M]."""
    _given(q, row_scale)
    (_native or binding()).quantize_int8(q, row_scale, x, stream)


def quantize_int8(x, stream=None):
    """Allocate and return (q int8 [M, K], row_scale float32 [M]): see quantize_int8_into."""
    return (_native or binding()).quantize_int8(None, None, x, stream)


def gemm_int8_into(y, q, row_scale, w: "WeightInt8", workspace=None, stream=None) -> None:
    """y[m, n] = (q[m] . w[n]) * row_scale[m] * channel_scale[n], the sum exact
    (y float16 or float32, preallocated; any number of rows)."""
    _given(y)
    (_native or binding()).gemm_int8(y, q, row_scale, w.codes, w.channel_scale, None, workspace, stream)


def gemm_int8(q, row_scale, w: "WeightInt8", out_dtype=None, workspace=None, stream=None):
    """Allocate y [M, N] (float16 unless out_dtype says otherwise): see gemm_int8_into."""
    return (_native or binding()).gemm_int8(None, q, row_scale, w.codes, w.channel_scale, out_dtype, workspace, stream)


def tile_device_error(clear: bool = True) -> int:
    """As device_error, for the experts' and int8 products."""
    v = ctypes.c_uint(0)
    _check(library().skinny_tile_device_error(1 if clear else 0, ctypes.byref(v)), "skinny_tile_device_error")
    return int(v.value)


# ---------------------------------------------------------------------------
# Verification of drafted tokens
# ---------------------------------------------------------------------------

def verify_draft_into(tokens, accepted, target, draft, draft_tokens, uniform, num_drafts=None, stream=None) -> None:
    """A verify round against the target's probabilities, from given random
    numbers: draft i of a request is accepted while uniform[i] * q_i(d_i) <
    p_i(d_i); the next token is drawn from max(p - q, 0) at the first draft that
    is not accepted, or from the last row of p, with uniform[S].

    target        [B, S+1, V] float32, float16 or bfloat16; unit stride along V
    draft         [B, S, V] of target's dtype, or None (drafts without a distribution)
    draft_tokens  int32 [B, S];  uniform  float32 [B, S+1] in [0, 1)
    num_drafts    int32 [B], or None for S each
    tokens        int32 [B, S+1]: accepted drafts, the drawn token, then -1
    accepted      int32 [B]
    """
    _given(tokens, accepted)
    (_native or binding()).verify_draft(tokens, accepted, target, draft, draft_tokens, uniform, num_drafts, stream)


def verify_draft(target, draft, draft_tokens, uniform, num_drafts=None, stream=None):
    """Allocate and return (tokens int32 [B, S+1], accepted int32 [B]): see verify_draft_into."""
    return (_native or binding()).verify_draft(None, None, target, draft, draft_tokens, uniform, num_drafts, stream)
