"""B200-native W4A16 weight-only matmul: thin Python binding of ``libw4a16.so``.

Every step of the computation runs in the library's sm_100a kernels; this
module only checks tensor metadata, passes device pointers and the current
CUDA stream, and turns status codes into exceptions.  PyTorch provides
device memory and streams.  There is no CPU fallback: without a CUDA device
or without the built library every call raises.  The calls of the 8-bit layer and
of the block norms go through a native module (``binding/w8_native.cpp``) that
does the same checks and allocations in C++.

Entry points (same names as the C ABI in ``include/w4a16.h``):

* :func:`w4_quantize_pack` -- bf16 W [N, K] -> packed int4 (int32 [N, K/8]),
  fp16 scales and zeros (``zero="float"``: fractional zero point;
  ``meta="bf16"``: bf16 scales and zeros)
* :func:`w4a16_gemm` -- Y = X . dequant(W)^T (or dX = dY . dequant(W) with
  ``transposed=True``), optional bias
* :func:`w4a16_gemv` -- the same for M <= 4 (TMA-streamed weights, exact
  products on the tensor pipe, fp32 sums)
* :func:`w4_gather_columns` / :func:`w4_scatter_columns` -- the column
  permutations of act-order weights (``perm=`` on the calls above)
* :func:`w8_quantize_rows` -- bf16 rows -> int8 codes and one fp32 scale per row
* :func:`w8a8_gemm` -- the product of int8 tokens and int8 weights with a scale
  for each token and channel, forward (optional bias) and transposed
* :func:`w8a8_linear` -- both on bf16 rows in one call
* :func:`w4_block_norm` / :func:`w4_block_norm_backward` -- the norms before and
  after a block fused with its gate, residual scale and residual add, as bf16 or
  as int8 rows for the products above
* :func:`w4_workspace_bytes`, :func:`w4_device_error`

:mod:`gemv_w4a16_groupwise_b200.tp` shards one layer over torch.distributed
ranks (column-parallel over N, row-parallel over K) on top of these calls.

``packed`` may also be given as its two-per-byte view, uint8 [N, K/2] (the
same bytes; the even k in the low nibble).
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Any, NamedTuple

from . import build as _build

W4_MODE_GLOBAL = 0
W4_MODE_ROWWISE = 1
W4_MODE_GROUPWISE = 2
MODES = {"global": W4_MODE_GLOBAL, "rowwise": W4_MODE_ROWWISE, "groupwise": W4_MODE_GROUPWISE}
W4_ZERO_FLOAT = 0x10
W4_META_BF16 = 0x20

_lock = threading.Lock()
_lib = None


class W4Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        msg = f"{what}: {library().w4_status_string(status).decode()}"
        if status == 5:
            msg += f" ({library().w4_last_cuda_error().decode()})"
        super().__init__(msg)


def library_path() -> str:
    return _build.LIB


def library():
    """Load (building first if needed) the in-tree CUDA library."""
    global _lib
    with _lock:
        if _lib is None:
            path = _build.build()
            lib = ctypes.CDLL(path)
            P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
            lib.w4_status_string.argtypes = [I]
            lib.w4_status_string.restype = ctypes.c_char_p
            lib.w4_quantize_workspace_bytes.argtypes = [I, I, I]
            lib.w4_quantize_workspace_bytes.restype = Z
            lib.w4_quantize_pack.argtypes = [P, I, I, I, I, P, P, P, P, Z, P]
            lib.w4_quantize_pack.restype = I
            lib.w4_workspace_bytes.argtypes = [I, I, I, I]
            lib.w4_workspace_bytes.restype = Z
            for name in ("w4a16_gemm", "w4a16_gemv"):
                f = getattr(lib, name)
                f.argtypes = [P, I, I, I, P, P, P, I, I, P, I, P, P, Z, P]
                f.restype = I
            lib.w4_device_error.argtypes = [ctypes.POINTER(I)]
            lib.w4_device_error.restype = I
            lib.w4_last_cuda_error.argtypes = []
            lib.w4_last_cuda_error.restype = ctypes.c_char_p
            lib.w4_launch_count.argtypes = []
            lib.w4_launch_count.restype = ctypes.c_uint64
            lib.w4_set_debug_checks.argtypes = [I]
            lib.w4_set_debug_checks.restype = I
            lib.w4_debug_set_wait_limit.argtypes = [ctypes.c_ulonglong]
            lib.w4_debug_set_wait_limit.restype = I
            lib.w4_debug_withhold_stage.argtypes = [I]
            lib.w4_debug_withhold_stage.restype = I
            lib.w4_gather_columns.argtypes = [P, I, I, P, I, P, P]
            lib.w4_gather_columns.restype = I
            lib.w4_scatter_columns.argtypes = [P, I, I, P, I, P, P]
            lib.w4_scatter_columns.restype = I
            lib.w4_invert_permutation.argtypes = [P, I, P, P]
            lib.w4_invert_permutation.restype = I
            L, F = ctypes.c_longlong, ctypes.c_float
            lib.w8_quantize_rows.argtypes = [P, I, I, P, P, L, P, P]
            lib.w8_quantize_rows.restype = I
            for name in ("w8a8_workspace_bytes", "w8a8_linear_workspace_bytes"):
                f = getattr(lib, name)
                f.argtypes = [I, I, I, I]
                f.restype = Z
            lib.w8a8_gemm.argtypes = [P, L, P, I, I, I, P, L, P, P, I, P, P, Z, P]
            lib.w8a8_gemm.restype = I
            lib.w8a8_linear.argtypes = [P, I, I, I, P, L, P, P, I, P, P, Z, P]
            lib.w8a8_linear.restype = I
            lib.w4_block_norm.argtypes = [P, P, I, I, P, P, I, F, P, F, F, P, P, L, P, P, P]
            lib.w4_block_norm.restype = I
            lib.w4_block_norm_workspace_bytes.argtypes = [I, I]
            lib.w4_block_norm_workspace_bytes.restype = Z
            lib.w4_block_norm_backward.argtypes = [P, P, P, P, P, I, I, P, P, I, F, P, F, P, P, P, P, P, P, Z, P]
            lib.w4_block_norm_backward.restype = I
            _lib = lib
    return _lib


def _torch():
    import torch
    return torch


def _mode(mode, zero: str = "int", meta: str = "fp16") -> int:
    """The C mode argument: base mode or-ed with the format flags."""
    m = MODES[mode] if isinstance(mode, str) else int(mode)
    if zero not in ("int", "float") or meta not in ("fp16", "bf16"):
        raise ValueError(f"zero must be 'int' or 'float' and meta 'fp16' or 'bf16', got {zero!r}, {meta!r}")
    return m | (W4_ZERO_FLOAT if zero == "float" else 0) | (W4_META_BF16 if meta == "bf16" else 0)


def _meta_dtype(meta: str):
    torch = _torch()
    return torch.bfloat16 if meta == "bf16" else torch.float16


def _check_cuda(t, name, dtype, shape=None):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device (no CPU path exists)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _packed_words(packed, N: int, K: int):
    """The packed codes as int32 [N, K/8]; a uint8 [N, K/2] two-per-byte view is
    reinterpreted (same bytes), anything else is passed on for the checks."""
    torch = _torch()
    if isinstance(packed, torch.Tensor) and packed.dtype == torch.uint8:
        if tuple(packed.shape) != (N, K // 2) or not packed.is_contiguous():
            raise ValueError(f"uint8 packed codes must be contiguous [{N}, {K // 2}]")
        return packed.view(torch.int32)
    return packed


def _check_perm(perm, K: int, dev):
    torch = _torch()
    _check_cuda(perm, "perm", torch.int32, (K,))
    if perm.device != dev:
        raise ValueError("perm must be on the activations' device")


def _device_index(device) -> int:
    torch = _torch()
    if isinstance(device, int):
        return device
    return device.index if device.index is not None else torch.cuda.current_device()


def _stream_ptr(device):
    """The current stream of `device` as a raw handle.  PyTorch's own raw
    accessor (what its compiled kernels use) costs a tenth of building the
    Stream object; the public call is the fallback."""
    torch = _torch()
    idx = _device_index(device)
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is not None:
        return ctypes.c_void_p(raw(idx))
    return ctypes.c_void_p(torch.cuda.current_stream(idx).cuda_stream)


class _OnDevice:
    """Make `idx` the current device for a library call and restore the
    previous one, switching only when they differ (the library launches on
    the current device)."""

    __slots__ = ("idx", "prev", "_get", "_set")

    def __init__(self, device):
        torch = _torch()
        self.idx = _device_index(device)
        self._get = getattr(torch._C, "_cuda_getDevice", None)
        self._set = getattr(torch._C, "_cuda_setDevice", None)
        self.prev = None

    def __enter__(self):
        if self._get is None or self._set is None:
            self.prev = _torch().cuda.device(self.idx)
            self.prev.__enter__()
            return self
        self.prev = self._get()
        if self.prev != self.idx:
            self._set(self.idx)
        return self

    def __exit__(self, *exc):
        if self._get is None or self._set is None:
            return self.prev.__exit__(*exc)
        if self.prev != self.idx:
            self._set(self.prev)
        return False


# w4_workspace_bytes by (device, M, N, K, transposed): a pure function of
# the shape and the device's SM count
_ws_cache: dict = {}


def meta_shape(N: int, K: int, mode, group_size: int):
    m = _mode(mode) & 0x0F
    if m == W4_MODE_GLOBAL:
        return (1, 1)
    if m == W4_MODE_ROWWISE:
        return (N, 1)
    if group_size <= 0 or K % group_size:
        raise ValueError(f"group_size {group_size} must divide K={K}")
    return (N, K // group_size)


def w4_quantize_workspace_bytes(N: int, K: int, mode) -> int:
    return int(library().w4_quantize_workspace_bytes(N, K, _mode(mode)))


def w4_workspace_bytes(M: int, N: int, K: int, transposed: bool = False) -> int:
    return int(library().w4_workspace_bytes(M, N, K, int(bool(transposed))))


def w4_quantize_pack(W, mode="groupwise", group_size: int = 128, out=None, zero: str = "int",
                     meta: str = "fp16", perm=None):
    """Quantize bf16 W [N, K] (CUDA) -> (packed int32 [N, K/8], scales, zeros).

    ``zero="float"`` keeps a fractional zero point (the HQQ-style quantizer);
    ``meta="bf16"`` stores scales and zeros as bf16 instead of fp16;
    ``perm`` (int32 [K], a permutation) quantizes W[:, perm] (act-order).
    """
    torch = _torch()
    _check_cuda(W, "W", torch.bfloat16)
    N, K = W.shape
    if perm is not None:
        _check_perm(perm, K, W.device)
        W = w4_gather_columns(W, perm)
    shape = meta_shape(N, K, mode, group_size)
    dev = W.device
    mdt = _meta_dtype(meta)
    if out is None:
        packed = torch.empty((N, K // 8), dtype=torch.int32, device=dev)
        scales = torch.empty(shape, dtype=mdt, device=dev)
        zeros = torch.empty(shape, dtype=mdt, device=dev)
    else:
        packed, scales, zeros = out
        _check_cuda(scales, "scales", mdt, shape)
        _check_cuda(zeros, "zeros", mdt, shape)
    nws = w4_quantize_workspace_bytes(N, K, mode)
    ws = torch.empty(max(nws, 16), dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        st = library().w4_quantize_pack(W.data_ptr(), N, K, _mode(mode, zero, meta), int(group_size),
                                        packed.data_ptr(), scales.data_ptr(), zeros.data_ptr(),
                                        ws.data_ptr(), nws, _stream_ptr(dev))
    if st != 0:
        raise W4Error(st, "w4_quantize_pack")
    return packed, scales, zeros


def _matmul(fname, A, packed, scales, zeros, mode, group_size, N, K, bias, transposed, out, zero,
            perm=None):
    torch = _torch()
    packed = _packed_words(packed, N, K)
    if perm is not None:
        # act-order: forward gathers X's columns; transposed scatters dX's
        _check_cuda(A, "A", torch.bfloat16)
        _check_perm(perm, K, A.device)
        if not transposed:
            return _matmul(fname, w4_gather_columns(A, perm), packed, scales, zeros, mode, group_size, N, K,
                           bias, False, out, zero)
        bias_p = None if bias is None else w4_gather_columns(bias.view(1, -1), perm).view(-1)
        part = _matmul(fname, A, packed, scales, zeros, mode, group_size, N, K, bias_p, True, None, zero)
        # dX[:, perm[j]] = part[:, j]: a gather by the inverse permutation
        return w4_gather_columns(part, w4_invert_permutation(perm), out=out)
    _check_cuda(A, "A", torch.bfloat16)
    _check_cuda(packed, "packed", torch.int32, (N, K // 8))
    # the metadata type follows the scales' dtype (fp16 or bf16)
    meta = "bf16" if isinstance(scales, torch.Tensor) and scales.dtype == torch.bfloat16 else "fp16"
    _check_cuda(scales, "scales", _meta_dtype(meta), meta_shape(N, K, mode, group_size))
    _check_cuda(zeros, "zeros", _meta_dtype(meta), meta_shape(N, K, mode, group_size))
    if A.dim() != 2:
        raise ValueError("A must be 2-D")
    M = A.shape[0]
    in_len, out_len = (N, K) if transposed else (K, N)
    if A.shape[1] != in_len:
        raise ValueError(f"A must have {in_len} columns, got {A.shape[1]}")
    if bias is not None:
        _check_cuda(bias, "bias", torch.bfloat16, (out_len,))
    dev = A.device
    if out is None:
        out = torch.empty((M, out_len), dtype=torch.bfloat16, device=dev)
    else:
        _check_cuda(out, "out", torch.bfloat16, (M, out_len))
    with _OnDevice(dev) as on:
        key = (on.idx, M, N, K, bool(transposed))
        nws = _ws_cache.get(key)
        if nws is None:
            nws = w4_workspace_bytes(M, N, K, transposed)
            if len(_ws_cache) > 4096:
                _ws_cache.clear()
            _ws_cache[key] = nws
        ws = torch.empty(nws, dtype=torch.uint8, device=dev) if nws else None
        st = getattr(library(), fname)(
            A.data_ptr(), M, N, K, packed.data_ptr(), scales.data_ptr(), zeros.data_ptr(),
            _mode(mode, zero, meta), int(group_size), None if bias is None else bias.data_ptr(),
            int(bool(transposed)), out.data_ptr(), None if ws is None else ws.data_ptr(), nws,
            _stream_ptr(on.idx))
    if st != 0:
        raise W4Error(st, fname)
    return out


def w4a16_gemm(A, packed, scales, zeros, mode="groupwise", group_size: int = 128, *, N: int,
               K: int, bias=None, transposed: bool = False, out=None, zero: str = "int", perm=None):
    """Y = A . dequant(W)^T  (A [M, K])  or, transposed, dX = A . dequant(W)  (A [M, N]).

    ``zero`` must name the quantizer's zero point ("int" or "float"); bf16 scales
    and zeros are recognised by their dtype; ``perm`` (int32 [K]) marks act-order
    weights whose packed column j is input channel perm[j]."""
    return _matmul("w4a16_gemm", A, packed, scales, zeros, mode, group_size, N, K, bias,
                   transposed, out, zero, perm)


def w4a16_gemv(A, packed, scales, zeros, mode="groupwise", group_size: int = 128, *, N: int,
               K: int, bias=None, transposed: bool = False, out=None, zero: str = "int", perm=None):
    """Small-batch (M <= 4) path of :func:`w4a16_gemm`: TMA-streamed weights, exact
    products on the tensor pipe with fp32 sums, forward and transposed."""
    return _matmul("w4a16_gemv", A, packed, scales, zeros, mode, group_size, N, K, bias,
                   transposed, out, zero, perm)


def w4_gather_columns(A, idx, out=None):
    """out[m, j] = A[m, idx[j]]: bf16 A [M, C] (CUDA), int32 idx [L] -> bf16 [M, L]."""
    torch = _torch()
    _check_cuda(A, "A", torch.bfloat16)
    _check_cuda(idx, "idx", torch.int32)
    if A.dim() != 2 or idx.dim() != 1:
        raise ValueError("A must be 2-D and idx 1-D")
    M, C = A.shape
    L = idx.shape[0]
    if out is None:
        out = torch.empty((M, L), dtype=torch.bfloat16, device=A.device)
    else:
        _check_cuda(out, "out", torch.bfloat16, (M, L))
    with torch.cuda.device(A.device):
        st = library().w4_gather_columns(A.data_ptr(), M, C, idx.data_ptr(), L, out.data_ptr(),
                                         _stream_ptr(A.device))
    if st != 0:
        raise W4Error(st, "w4_gather_columns")
    return out


def w4_invert_permutation(perm, out=None):
    """inv [n] with inv[perm[j]] = j (int32, CUDA; perm a permutation of [0, n))."""
    torch = _torch()
    _check_cuda(perm, "perm", torch.int32)
    n = perm.shape[0]
    inv = torch.empty_like(perm) if out is None else out
    with torch.cuda.device(perm.device):
        st = library().w4_invert_permutation(perm.data_ptr(), n, inv.data_ptr(), _stream_ptr(perm.device))
    if st != 0:
        raise W4Error(st, "w4_invert_permutation")
    return inv


def w4_scatter_columns(A, idx, dst_cols: int, out=None):
    """out[m, idx[j]] = A[m, j]: bf16 A [M, L], int32 idx [L] (no repeats) -> bf16
    [M, dst_cols] (a fresh tensor, zero where no index lands, unless `out` is given)."""
    torch = _torch()
    _check_cuda(A, "A", torch.bfloat16)
    _check_cuda(idx, "idx", torch.int32)
    M, L = A.shape
    if idx.shape != (L,):
        raise ValueError(f"idx must have shape ({L},)")
    if out is None:
        out = torch.zeros((M, dst_cols), dtype=torch.bfloat16, device=A.device)
    else:
        _check_cuda(out, "out", torch.bfloat16, (M, dst_cols))
    with torch.cuda.device(A.device):
        st = library().w4_scatter_columns(A.data_ptr(), M, L, idx.data_ptr(), dst_cols, out.data_ptr(),
                                          _stream_ptr(A.device))
    if st != 0:
        raise W4Error(st, "w4_scatter_columns")
    return out


# The 8-bit layer's and the block norms' calls take a few microseconds of
# device time on a few tokens, less than Python needs for their checks and
# tensors.  An ordinary call is made by the native module (binding/
# w8_native.cpp) in one C function; where that finds an argument it does not
# take (None), the call goes through the checks here, which say what is wrong.
class _NoNative:
    """In place of the native module where it cannot be had: takes no call, so the Python checks make
    each of them, on the same kernels."""
    @staticmethod
    def _none(*args):
        return None

    quantize_rows = gemm = linear = norm = norm_backward = _none


def _load_native():
    import importlib.machinery
    import importlib.util
    import subprocess
    import warnings
    try:
        loader = importlib.machinery.ExtensionFileLoader("w8_native", _build.build_binding())
        native = importlib.util.module_from_spec(importlib.util.spec_from_loader("w8_native", loader))
        loader.exec_module(native)
    except (OSError, ImportError, subprocess.CalledProcessError) as e:
        warnings.warn(f"the binding's native part could not be built or loaded ({e}); calls of the 8-bit layer and "
                      "of the block norms go through Python and take a few microseconds more", RuntimeWarning)
        return _NoNative
    lib = library()
    native.bind(*(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in (
        "w8_quantize_rows", "w8a8_workspace_bytes", "w8a8_linear_workspace_bytes", "w8a8_gemm", "w8a8_linear",
        "w4_block_norm", "w4_block_norm_workspace_bytes", "w4_block_norm_backward")), BlockNorm, BlockNormGrad)
    return native


class _Torch:
    """torch, what the calls below use of it, and the native calls, looked up once."""
    lock = threading.Lock()      # not the library's, which is taken inside
    torch = None                 # set last: what reads it without the lock finds the rest
    native = None

    @classmethod
    def load(cls):
        with cls.lock:
            if cls.torch is None:
                cls._load()

    @classmethod
    def _load(cls):
        torch = _torch()
        cls.native = _load_native()
        cls.bf16, cls.f32, cls.i8, cls.u8 = torch.bfloat16, torch.float32, torch.int8, torch.uint8
        cls.empty_like = torch.empty_like
        cls.get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        cls.stream = raw or (lambda idx: torch.cuda.current_stream(idx).cuda_stream)
        cls.lib = library()
        cls.torch = torch


def _native():
    if _Torch.torch is None:
        _Torch.load()
    return _Torch.native


def _call(name, dev, *args):
    """The library call on device `dev` and its current stream."""
    f = getattr(_Torch.lib, name)
    if _Torch.get_device() == dev:
        st = f(*args, _Torch.stream(dev))
    else:
        with _OnDevice(dev):
            st = f(*args, _Torch.stream(dev))
    if st != 0:
        raise W4Error(st, name)


def _check_rows(t, name, dtype, dev, shape):
    """A dense tensor of this dtype and shape on CUDA device `dev`."""
    if (t.__class__ is _Torch.torch.Tensor and t.dtype is dtype and t.get_device() == dev and t.shape == shape
            and t.is_contiguous()):
        return
    _check_cuda(t, name, dtype, shape)
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")


def _check_first(t, name):
    """The bf16 matrix that a call is about; returns its device's index."""
    if _Torch.torch is None:
        _Torch.load()
    if t.__class__ is _Torch.torch.Tensor and t.dtype is _Torch.bf16 and t.dim() == 2 and t.is_contiguous():
        dev = t.get_device()
        if dev >= 0:
            return dev
    _check_cuda(t, name, _Torch.bf16)
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    return t.get_device()


def _check_codes(t, name, dev=None, rows=None, cols=None) -> int:
    """Check int8 rows and return their stride in bytes, a multiple of 16 that
    covers a row rounded up to 16 (the layout :func:`w8_quantize_rows` gives)."""
    if t.__class__ is _Torch.torch.Tensor and t.dtype is _Torch.i8 and t.dim() == 2 and t.get_device() == dev:
        R, C = t.shape
        ld, one = t.stride()
        if R > 1 and C % 16 == 0 and one == 1 and ld % 16 == 0 and ld >= C and rows is None:
            return ld
    torch = _Torch.torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device (no CPU path exists)")
    if t.dtype != torch.int8:
        raise TypeError(f"{name} must be {torch.int8}, got {t.dtype}")
    if dev is not None and t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
    if t.dim() != 2 or (rows is not None and tuple(t.shape) != (rows, cols)):
        raise ValueError(f"{name} must be 2-D{'' if rows is None else f' of shape {(rows, cols)}'}, "
                         f"got {tuple(t.shape)}")
    R, C = t.shape
    need = (C + 15) // 16 * 16
    ld = t.stride(0) if R > 1 else need
    if (C > 1 and t.stride(1) != 1) or ld % 16 or ld < need:
        raise ValueError(f"{name}: rows must be dense and start every multiple of 16 bytes, got strides {t.stride()}")
    if R and t.untyped_storage().nbytes() < t.storage_offset() + (R - 1) * ld + need:
        raise ValueError(f"{name}: the last row must be readable up to a multiple of 16 bytes")
    return ld


def _empty_codes(like, R: int, C: int):
    C16 = (C + 15) // 16 * 16
    q = like.new_empty(R, C16, dtype=_Torch.i8)
    return q if C16 == C else q[:, :C]


def w8_quantize_rows(X, channel_scales=None, out=None):
    """int8 codes and one fp32 scale per row of bf16 X [R, C]: scales = max|v| / 127,
    codes = rint(127 v / max|v|), v = X, or X * channel_scales (fp32 [C]).

    The codes' rows start every multiple of 16 bytes (a view of a wider tensor
    when C is not one).  A row of zeros has scale 0, a row with an infinity or a
    NaN scale NaN and codes 0.  ``out``: (codes, scales) to write into."""
    if out is None:
        r = _native().quantize_rows(X, channel_scales)
        if r.__class__ is tuple:
            return r
        if r is not None:
            raise W4Error(r, "w8_quantize_rows")
    dev = _check_first(X, "X")
    R, C = X.shape
    if channel_scales is not None:
        _check_rows(channel_scales, "channel_scales", _Torch.f32, dev, (C,))
    if out is None:
        codes, scales = _empty_codes(X, R, C), X.new_empty(R, dtype=_Torch.f32)
        ld = (C + 15) // 16 * 16
    else:
        codes, scales = out
        ld = _check_codes(codes, "codes", dev, R, C)
        _check_rows(scales, "scales", _Torch.f32, dev, (R,))
    _call("w8_quantize_rows", dev, X.data_ptr(), R, C, _ptr(channel_scales), codes.data_ptr(), ld, scales.data_ptr())
    return codes, scales


def _w8_operands(A, dev, codes, scales, bias, transposed, out):
    """Checks that w8a8_gemm and w8a8_linear share; returns (M, N, K, stride of the weights, output)."""
    ldw = _check_codes(codes, "codes", dev)
    N, K = codes.shape
    in_len, out_len = (N, K) if transposed else (K, N)
    M, got = A.shape
    if got != in_len:
        raise ValueError(f"A must have {in_len} columns, got {got}")
    if scales is not None:
        _check_rows(scales, "scales", _Torch.f32, dev, (N,))
    if bias is not None:
        _check_rows(bias, "bias", _Torch.bf16, dev, (out_len,))
    if out is None:
        out = A.new_empty(M, out_len, dtype=_Torch.bf16)
    else:
        _check_rows(out, "out", _Torch.bf16, dev, (M, out_len))
    return M, N, K, ldw, out


def _scratch(query, dev, like, *shape):
    """Scratch of the size that the library asks for (a pure function of the shape and the device)."""
    key = (query, dev, *shape)
    n = _ws_cache.get(key)
    if n is None:
        with _OnDevice(dev):
            n = int(getattr(_Torch.lib, query)(*shape))
        if len(_ws_cache) > 4096:
            _ws_cache.clear()
        _ws_cache[key] = n
    return (like.new_empty(n, dtype=_Torch.u8) if n else None), n


def w8a8_gemm(A, a_scales, codes, scales=None, *, bias=None, transposed: bool = False, out=None):
    """Product of int8 tokens A with int8 weights ``codes`` [N, K], exact integer sums:

    Y[m, n] = a_scales[m] scales[n] sum_k A[m, k] codes[n, k] + bias[n], or, transposed,
    dX[m, k] = a_scales[m] sum_n A[m, n] codes[n, k] + bias[k], where A holds the rows of
    dY quantized with ``channel_scales=scales`` and ``scales`` is left out here.
    bf16 output; ``out`` may not overlap the inputs."""
    r = _native().gemm(A, a_scales, codes, scales, bias, transposed, out)
    if r is not None:
        if r.__class__ is int:
            raise W4Error(r, "w8a8_gemm")
        return r
    tr = 1 if transposed else 0
    if tr and scales is not None:
        raise ValueError("transposed: fold the weights' scales into A "
                         "(w8_quantize_rows with channel_scales) and pass scales=None")
    if not tr and scales is None:
        raise ValueError("scales of the weights are needed")
    if a_scales is None:
        raise ValueError("a_scales are needed")
    dev = A.get_device() if isinstance(A, _Torch.torch.Tensor) and A.is_cuda else None
    lda = _check_codes(A, "A", dev)
    M, N, K, ldw, out = _w8_operands(A, dev, codes, scales, bias, tr, out)
    _check_rows(a_scales, "a_scales", _Torch.f32, dev, (M,))
    ws, nws = _scratch("w8a8_workspace_bytes", dev, out, M, N, K, tr)
    _call("w8a8_gemm", dev, A.data_ptr(), lda, a_scales.data_ptr(), M, N, K, codes.data_ptr(), ldw, _ptr(scales),
          _ptr(bias), tr, out.data_ptr(), _ptr(ws), nws)
    return out


def w8a8_linear(A, codes, scales, *, bias=None, transposed: bool = False, out=None):
    """8-bit linear layer on bf16 rows: :func:`w8_quantize_rows` on A and
    :func:`w8a8_gemm` in one call.  Y = A . dequant(codes)^T (A [M, K]), or,
    transposed, dX = A . dequant(codes) (A [M, N]).  ``out`` may not overlap the inputs.
    ``scales`` start on 16 bytes here; those of the two calls may be slices that do not,
    but for ``channel_scales``."""
    r = _native().linear(A, codes, scales, bias, transposed, out)
    if r is not None:
        if r.__class__ is int:
            raise W4Error(r, "w8a8_linear")
        return r
    dev = _check_first(A, "A")
    if scales is None:
        raise ValueError("scales of the weights are needed")
    tr = 1 if transposed else 0
    M, N, K, ldw, out = _w8_operands(A, dev, codes, scales, bias, tr, out)
    ws, nws = _scratch("w8a8_linear_workspace_bytes", dev, out, M, N, K, tr)
    _call("w8a8_linear", dev, A.data_ptr(), M, N, K, codes.data_ptr(), ldw, scales.data_ptr(), _ptr(bias), tr,
          out.data_ptr(), _ptr(ws), nws)
    return out


class BlockNorm(NamedTuple):
    """What :func:`w4_block_norm` gives; fields that were not asked for are None."""
    residual: Any       # bf16 [M, C]
    normed: Any         # bf16 [M, C], or int8 codes
    scales: Any         # fp32 [M], of the codes
    rstd: Any           # fp32 [2, M], for the backward pass


class BlockNormGrad(NamedTuple):
    """Gradients of :func:`w4_block_norm`; None where the forward had no such input."""
    d_x: Any
    d_y: Any
    d_pre_weight: Any
    d_post_weight: Any
    d_gate: Any


def _check_norm(M, C, dev, pre_weight, post_weight, gate, y):
    """The norm's weights and gate; returns the C API's gate kind."""
    bf16 = _Torch.bf16
    _check_rows(pre_weight, "pre_weight", bf16, dev, (C,))
    if y is not None:
        _check_rows(y, "y", bf16, dev, (M, C))
    elif post_weight is not None or gate is not None:
        raise ValueError("post_weight and gate belong to y, which is not given")
    if post_weight is not None:
        _check_rows(post_weight, "post_weight", bf16, dev, (C,))
    if gate is None:
        return 0
    if isinstance(gate, _Torch.torch.Tensor) and gate.dim() == 1:
        _check_rows(gate, "gate", bf16, dev, (C,))
        return 1
    _check_rows(gate, "gate", bf16, dev, (M, C))
    return 2


def _ptr(t):
    return None if t is None else t.data_ptr()


def w4_block_norm(x, y=None, *, pre_weight, post_weight=None, gate=None, residual_scale: float = 1.0,
                  weight_offset: float = 0.0, eps: float = 1e-5, quantize: bool = False,
                  keep_rstd: bool = False, residual_out=None) -> BlockNorm:
    """residual = x + residual_scale * gate * norm(y; post_weight), then norm(residual; pre_weight).

    x, y: bf16 [M, C], C <= 16384; y is the output of the block before (None: there is
    none, and x itself is normed and returned as the residual).  post_weight (bf16 [C])
    is the norm after that block, pre_weight the one before the next; weights are
    w + weight_offset.  gate: bf16 [C] or [M, C].  ``quantize`` gives the normed rows as
    int8 codes and scales for :func:`w8a8_gemm` instead of bf16.  ``keep_rstd`` keeps what
    :func:`w4_block_norm_backward` needs.  ``residual_out`` may be x or y (in place).
    A row's result does not depend on the others; with an odd C its last bits may differ
    between an even and an odd place (rows there begin at either half of a word)."""
    r = _native().norm(x, y, pre_weight, post_weight, gate, residual_scale, weight_offset, eps, quantize, keep_rstd,
                       residual_out)
    if r is not None:
        if r.__class__ is int:
            raise W4Error(r, "w4_block_norm")
        return r
    dev = _check_first(x, "x")
    M, C = x.shape
    kind = _check_norm(M, C, dev, pre_weight, post_weight, gate, y)
    if y is None:
        if residual_out is not None:
            raise ValueError("without y the residual is x itself")
        residual = x
    elif residual_out is None:
        residual = _Torch.empty_like(x)
    else:
        _check_rows(residual_out, "residual_out", _Torch.bf16, dev, (M, C))
        residual = residual_out
    if quantize:
        normed, scales = _empty_codes(x, M, C), x.new_empty(M, dtype=_Torch.f32)
    else:
        normed, scales = _Torch.empty_like(x), None
    rstd = x.new_empty(2, M, dtype=_Torch.f32) if keep_rstd else None
    _call("w4_block_norm", dev, x.data_ptr(), _ptr(y), M, C, _ptr(post_weight), _ptr(gate), kind, residual_scale,
          pre_weight.data_ptr(), weight_offset, eps, None if y is None else residual.data_ptr(), normed.data_ptr(),
          (C + 15) // 16 * 16, _ptr(scales), _ptr(rstd))
    return BlockNorm(residual, normed, scales, rstd)


def w4_block_norm_backward(d_normed, residual, rstd, y=None, *, d_residual=None, pre_weight, post_weight=None,
                           gate=None, residual_scale: float = 1.0, weight_offset: float = 0.0) -> BlockNormGrad:
    """Gradients of :func:`w4_block_norm` from d_normed and d_residual (None: zero), with
    the residual and rstd that it returned (``keep_rstd=True``), its y, weights and gate.

    All bf16: d_x, d_y [M, C], d_pre_weight, d_post_weight [C], d_gate in the gate's shape.
    Quantized rows count as the values they stand for.  The same inputs give the same bits
    (a row by itself those of its place, as in the forward pass)."""
    r = _native().norm_backward(d_normed, residual, rstd, d_residual, y, pre_weight, post_weight, gate, residual_scale,
                                weight_offset)
    if r is not None:
        if r.__class__ is int:
            raise W4Error(r, "w4_block_norm_backward")
        return r
    dev = _check_first(d_normed, "d_normed")
    M, C = d_normed.shape
    bf16, empty_like = _Torch.bf16, _Torch.empty_like
    _check_rows(residual, "residual", bf16, dev, (M, C))
    _check_rows(rstd, "rstd", _Torch.f32, dev, (2, M))
    if d_residual is not None:
        _check_rows(d_residual, "d_residual", bf16, dev, (M, C))
    kind = _check_norm(M, C, dev, pre_weight, post_weight, gate, y)
    d_x = empty_like(d_normed)
    d_y = None if y is None else empty_like(y)
    d_pre = empty_like(pre_weight)
    d_post = None if post_weight is None else empty_like(post_weight)
    d_gate = None if gate is None else empty_like(gate)
    ws, nws = _scratch("w4_block_norm_workspace_bytes", dev, d_x, M, C)
    _call("w4_block_norm_backward", dev, d_normed.data_ptr(), _ptr(d_residual), residual.data_ptr(), rstd.data_ptr(),
          _ptr(y), M, C, _ptr(post_weight), _ptr(gate), kind, residual_scale, pre_weight.data_ptr(), weight_offset,
          d_x.data_ptr(), _ptr(d_y), d_pre.data_ptr(), _ptr(d_post), _ptr(d_gate), _ptr(ws), nws)
    return BlockNormGrad(d_x, d_y, d_pre, d_post, d_gate)


def w4_launch_count() -> int:
    """Kernel launches issued by the library in this process (host counter)."""
    return int(library().w4_launch_count())


def w4_set_debug_checks(on: bool) -> None:
    """Debug mode: w4_quantize_pack rejects NaN / Inf weights (W4_ERR_INVALID_ARG)."""
    library().w4_set_debug_checks(1 if on else 0)


def w4_debug_set_wait_limit(ns: int) -> None:
    """Limit of a kernel's bounded waits on the current device (0 = the default 2 s)."""
    st = library().w4_debug_set_wait_limit(int(ns))
    if st != 0:
        raise W4Error(st, "w4_debug_set_wait_limit")


def w4_debug_withhold_stage(stage: int) -> None:
    """Failure injection: the GEMV producers skip stage `stage` (-1: none)."""
    st = library().w4_debug_withhold_stage(int(stage))
    if st != 0:
        raise W4Error(st, "w4_debug_withhold_stage")


def w4_device_error() -> int:
    """Read and clear the device error word (synchronizes); 0 = no kernel gave up."""
    code = ctypes.c_int(0)
    st = library().w4_device_error(ctypes.byref(code))
    if st not in (0, 1, 6) or (st == 1 and code.value == 0):
        raise W4Error(st, "w4_device_error")
    return int(code.value)
