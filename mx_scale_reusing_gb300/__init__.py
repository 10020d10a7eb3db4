"""libmxnorm Python binding: argument marshalling over the C ABI.

Every step of the computation runs in the CUDA library (libmxnorm.so, built
in-tree by ``mx_scale_reusing_gb300._build``); this module only checks
tensors, allocates outputs with torch and passes raw device pointers plus the
current CUDA stream.  There is no CPU fallback: without the built library
every call raises ``MXNormLibraryMissing``.

A call runs on its `stream` argument, or on the device's current stream, and
the caller orders its inputs there.  What the call allocates belongs to that
stream's pool and, with `stream` given, is safe on the current stream as well;
on a third stream it needs Tensor.record_stream as any tensor does.

Method: "MXNorm: Reusing MXFP block scales for efficient tensor
normalisation", Resumen tecnico, 2. Metodologia ("Fundamentos Teoricos":
inverse RMS from the power mean of the MX block scales; "Implementacion":
one fused pass).  The function names follow the C ABI in include/mxnorm.h.
"""
from __future__ import annotations

import ctypes
import os

__all__ = [
    "FMT", "VARIANT", "MXNormError", "MXNormLibraryMissing", "lib", "library_path",
    "mxnorm_quant_fwd", "quant_fwd", "quant_fwd_host", "rmsnorm_mxfp8_ref_fwd", "device_errors",
    "code_bytes", "bwd_ste", "quant_fwd_nvfp4", "absmax", "nvfp4_tensor_scale", "quant_fwd_mma", "mx_cast",
    "linear_fwd", "mma_scale_bytes", "tiled_wait_drill", "mx_cast_fp4", "nvfp4_tensor_scale_gain",
    "quant_fwd_nvfp4_mma", "mx_dequant", "linear_fwd_fp4", "bwd_ste_ckpt", "linear_wgrad_ckpt",
    "linear_fp4_wait_drill", "linear_wgrad_wait_drill",
]

FMT = {"mxfp8": 0, "mxfp4": 1, "mxfp4_h16": 2, "mxfp8_h16": 3, "mxfp4_h32": 4, "mxfp8_h32": 5}
VARIANT = {"auto": 0, "warp_row": 1, "tiled_tma": 2}
STATUS = {0: "MXNORM_OK", 1: "MXNORM_ERR_INVALID_ARG", 2: "MXNORM_ERR_UNSUPPORTED",
          3: "MXNORM_ERR_MISALIGNED", 4: "MXNORM_ERR_CUDA"}

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "libmxnorm.so")
_lib = None


class MXNormLibraryMissing(RuntimeError):
    """libmxnorm.so is not built: every call raises this (there is no CPU
    fallback)."""


class MXNormError(RuntimeError):
    """A C-ABI call returned a non-zero mxnorm_status; `status` holds it and
    the message is the library's mxnorm_last_error() text."""

    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


def lib() -> ctypes.CDLL:
    """The loaded C library (raises MXNormLibraryMissing if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(library_path):
        raise MXNormLibraryMissing(
            f"{library_path} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'`")
    L = ctypes.CDLL(library_path)
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    L.mxnorm_quant_fwd.argtypes = [vp, i64, i64, i32, i32, vp, vp, vp, vp]
    L.mxnorm_quant_fwd.restype = i32
    L.mxnorm_quant_fwd_ex.argtypes = [vp, i64, i64, i32, i32, vp, vp, vp, i32, vp]
    L.mxnorm_quant_fwd_ex.restype = i32
    L.rmsnorm_mxfp8_ref_fwd.argtypes = [vp, i64, i64, ctypes.c_float, vp, vp, vp, vp, vp]
    L.rmsnorm_mxfp8_ref_fwd.restype = i32
    L.mxnorm_status_string.argtypes = [i32]
    L.mxnorm_status_string.restype = ctypes.c_char_p
    L.mxnorm_last_error.argtypes = []
    L.mxnorm_last_error.restype = ctypes.c_char_p
    L.mxnorm_abi_version.restype = i32
    L.mxnorm_quant_fwd_nvfp4.argtypes = [vp, i64, i64, i32, ctypes.c_float, vp, vp, vp, vp]
    L.mxnorm_quant_fwd_nvfp4.restype = i32
    L.mxnorm_absmax_bf16.argtypes = [vp, i64, vp, vp]
    L.mxnorm_absmax_bf16.restype = i32
    L.mxnorm_quant_fwd_nvfp4_dev.argtypes = [vp, i64, i64, i32, vp, vp, vp, vp, vp]
    L.mxnorm_quant_fwd_nvfp4_dev.restype = i32
    L.mxnorm_nvfp4_tensor_scale.argtypes = [vp, i64, vp, vp]
    L.mxnorm_nvfp4_tensor_scale.restype = i32
    L.mxnorm_bwd_ste.argtypes = [vp, vp, vp, i64, i64, vp, vp]
    L.mxnorm_mma_scale_bytes.argtypes = [i64, i64]
    L.mxnorm_mma_scale_bytes.restype = i64
    L.mxnorm_quant_fwd_layout.argtypes = [vp, i64, i64, i32, i32, vp, vp, vp, i32, vp]
    L.mxnorm_quant_fwd_layout.restype = i32
    L.mx_cast_fwd.argtypes = [vp, i64, i64, i32, vp, vp, i32, vp]
    L.mx_cast_fwd.restype = i32
    L.mx_cast_gain_fwd.argtypes = [vp, i64, i64, vp, ctypes.c_float, vp, vp, i32, vp]
    L.mx_cast_gain_fwd.restype = i32
    L.mxnorm_linear_fwd.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, vp, vp]
    L.mxnorm_linear_fwd.restype = i32
    L.mxnorm_bwd_ste.restype = i32
    L.mxnorm_tiled_wait_drill.argtypes = [vp, i64, i64, vp, vp, vp, i64, i64, vp]
    L.mxnorm_tiled_wait_drill.restype = i32
    L.mxnorm_mma_scale_bytes_fmt.argtypes = [i64, i64, i32]
    L.mxnorm_mma_scale_bytes_fmt.restype = i64
    L.mxnorm_quant_fwd_nvfp4_layout.argtypes = [vp, i64, i64, i32, vp, vp, vp, vp, i32, vp]
    L.mxnorm_quant_fwd_nvfp4_layout.restype = i32
    L.mx_cast_fp4_fwd.argtypes = [vp, i64, i64, i32, vp, ctypes.c_float, vp, vp, vp, i32, vp]
    L.mx_cast_fp4_fwd.restype = i32
    L.mxnorm_nvfp4_tensor_scale_gain.argtypes = [vp, i64, i64, vp, ctypes.c_float, vp, vp]
    L.mxnorm_nvfp4_tensor_scale_gain.restype = i32
    L.mxnorm_absmax_gain_bf16.argtypes = [vp, i64, i64, vp, ctypes.c_float, vp, vp]
    L.mxnorm_absmax_gain_bf16.restype = i32
    L.mx_dequant_fwd.argtypes = [vp, vp, i64, i64, i32, i32, vp, vp, vp]
    L.mx_dequant_fwd.restype = i32
    L.mxnorm_linear_fp4_fwd.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i32, vp, vp, vp, vp]
    L.mxnorm_linear_fp4_fwd.restype = i32
    L.mxnorm_linear_fp4_wait_drill.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i32, vp, vp, vp, i64, i64, vp]
    L.mxnorm_linear_fp4_wait_drill.restype = i32
    L.mxnorm_bwd_ste_ckpt.argtypes = [vp, vp, i32, vp, vp, i64, i64, vp, vp]
    L.mxnorm_bwd_ste_ckpt.restype = i32
    L.mxnorm_linear_wgrad_workspace_bytes.argtypes = [i64, i64, i64]
    L.mxnorm_linear_wgrad_workspace_bytes.restype = i64
    L.mxnorm_linear_wgrad_ckpt.argtypes = [vp, vp, i32, vp, vp, i64, i64, i64, vp, vp, i64, vp]
    L.mxnorm_linear_wgrad_ckpt.restype = i32
    L.mxnorm_linear_wgrad_wait_drill.argtypes = [vp, vp, i32, vp, vp, i64, i64, i64, vp, vp, i64, i32, i64, i64, vp]
    L.mxnorm_linear_wgrad_wait_drill.restype = i32
    L.mxnorm_device_errors.argtypes = [ctypes.POINTER(ctypes.c_uint32), i32]
    L.mxnorm_device_errors.restype = i32
    _lib = L
    return L


def _check(status: int):
    if status != 0:
        raise MXNormError(status, lib().mxnorm_last_error().decode())


def code_bytes(H: int, fmt: str) -> int:
    """Bytes of codes per row of H elements: one per E4M3 code, one per two
    E2M1 codes."""
    return H if fmt.startswith("mxfp8") else H // 2


def _stream_ptr(device, stream):
    """The raw cudaStream_t of `stream`, or of the device's current stream
    (looked up without building a Stream object: 0.1 us instead of 2)."""
    if stream is not None:
        return stream.cuda_stream
    import torch
    return torch._C._cuda_getCurrentRawStream(device.index)


class _Here:
    """The context of a call on the device that is current already."""

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return False


_here = _Here()


def _device(device):
    """Makes `device` current for a call; nothing to do (and 1.2 us less)
    where it is."""
    import torch
    return _here if torch.cuda.current_device() == device.index else torch.cuda.device(device)


def _workspace(shape, dtype, device, stream):
    """Memory from the pool of the stream that will use it (`stream`, or the current one)."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):  # anything that names a cudaStream_t
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _empty(shape, dtype, device, stream):
    """An output from the pool of the stream that will write it.  With a
    `stream` argument the current stream is recorded too: it usually reads
    the output once it has waited for `stream`, and the memory is not used
    again before both are done with it."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    t = _workspace(shape, dtype, device, stream)
    current = torch.cuda.current_stream(device)
    if current != stream:
        t.record_stream(current)
    return t


def _launch(fn, device, stream, *args):
    """Status-checked C call fn(*args, stream) with `device` current, on
    `stream` or the device's current one."""
    import torch
    sp = torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream
    if torch._C._cuda_getDevice() == device.index:
        status = fn(*args, sp)
    else:
        with torch.cuda.device(device):
            status = fn(*args, sp)
    if status != 0:
        _check(status)


def _require(t, name: str, device, dtype=None, min_numel: int = 0, byte_elems: bool = False):
    """Raise ValueError unless t is a contiguous CUDA tensor on `device` with
    dtype `dtype` (or 1-byte elements when byte_elems) and at least
    min_numel elements: the C ABI takes bare pointers and cannot check how
    large a buffer is."""
    if not (getattr(t, "is_cuda", False) and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if byte_elems and t.element_size() != 1:
        raise ValueError(f"{name} must have 1-byte elements (uint8 or an 8-bit float)")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call's tensors are on {device}")
    if t.numel() < min_numel:
        raise ValueError(f"{name} holds {t.numel()} elements, the call writes or reads {min_numel}")


def _need(t, name: str, index: int, n: int, dtype=None):
    """_require for the calls where host time counts: tensor t on CUDA device
    `index`, contiguous, at least n elements of dtype (None: 1-byte ones); the
    message of a refusal is _require's."""
    import torch
    if (not isinstance(t, torch.Tensor) or t.get_device() != index or not t.is_contiguous() or t.numel() < n
            or (t.dtype != dtype if dtype is not None else t.element_size() != 1)):
        _require(t, name, torch.device("cuda", max(0, index)), dtype, n, byte_elems=dtype is None)
        raise ValueError(f"{name} must be a contiguous CUDA tensor")


def mxnorm_quant_fwd(x_ptr: int, T: int, H: int, p: int, fmt: int, codes_ptr: int, scales_ptr: int,
                     inv_rms_ptr: int, stream_ptr: int = 0, variant: int = 0) -> None:
    """Raw C-ABI call on device pointers (ints); raises MXNormError."""
    _check(lib().mxnorm_quant_fwd_ex(x_ptr, T, H, p, fmt, codes_ptr, scales_ptr, inv_rms_ptr,
                                     variant, stream_ptr))


def quant_fwd(x, p: int = 2, fmt: str = "mxfp8", variant: str = "auto", out=None, stream=None):
    """MXNorm forward of a contiguous bf16 CUDA tensor x [..., H].

    Returns (codes uint8 [..., H or H/2], scales uint8 [..., H/32],
    inv_rms float32 [...]).  `out` may pass preallocated tensors in that
    order.  Runs on `stream` (default: the current stream); asynchronous.
    """
    import torch
    if not (x.is_cuda and x.dtype == torch.bfloat16 and x.is_contiguous()):
        raise ValueError("x must be a contiguous bfloat16 CUDA tensor")
    H = x.shape[-1]
    T = x.numel() // H if H else 0
    lead = tuple(x.shape[:-1])
    if out is None:
        codes = _empty(lead + (code_bytes(H, fmt),), torch.uint8, x.device, stream)
        scales = _empty(lead + (H // 32,), torch.uint8, x.device, stream)
        inv = _empty(lead, torch.float32, x.device, stream)
    else:
        codes, scales, inv = out
        _require(codes, "codes", x.device, min_numel=T * code_bytes(H, fmt), byte_elems=True)
        _require(scales, "scales", x.device, min_numel=T * (H // 32), byte_elems=True)
        _require(inv, "inv_rms", x.device, torch.float32, T)
    with _device(x.device):
        _check(lib().mxnorm_quant_fwd_ex(x.data_ptr(), T, H, int(p), FMT[fmt], codes.data_ptr(),
                                         scales.data_ptr(), inv.data_ptr(), VARIANT[variant],
                                         _stream_ptr(x.device, stream)))
    return codes, scales, inv


def rmsnorm_mxfp8_ref_fwd(x, eps: float = 1e-5, out=None, stream=None):
    """Two-pass RMSNorm-then-MXFP8 baseline.  Returns (y bf16 workspace,
    codes uint8, scales uint8, inv_rms float32)."""
    import torch
    if not (x.is_cuda and x.dtype == torch.bfloat16 and x.is_contiguous()):
        raise ValueError("x must be a contiguous bfloat16 CUDA tensor")
    H = x.shape[-1]
    T = x.numel() // H if H else 0
    lead = tuple(x.shape[:-1])
    if out is None:
        y = _empty(tuple(x.shape), torch.bfloat16, x.device, stream)
        codes = _empty(lead + (H,), torch.uint8, x.device, stream)
        scales = _empty(lead + (H // 32,), torch.uint8, x.device, stream)
        inv = _empty(lead, torch.float32, x.device, stream)
    else:
        y, codes, scales, inv = out
        _require(y, "y", x.device, torch.bfloat16, T * H)
        _require(codes, "codes", x.device, min_numel=T * H, byte_elems=True)
        _require(scales, "scales", x.device, min_numel=T * (H // 32), byte_elems=True)
        _require(inv, "inv_rms", x.device, torch.float32, T)
    with _device(x.device):
        _check(lib().rmsnorm_mxfp8_ref_fwd(x.data_ptr(), T, H, float(eps), y.data_ptr(), codes.data_ptr(),
                                           scales.data_ptr(), inv.data_ptr(), _stream_ptr(x.device, stream)))
    return y, codes, scales, inv


def absmax(x, stream=None, gamma=None, c: float = 1.0):
    """max |x| of a contiguous bf16 CUDA tensor, as a 1-element float32 CUDA
    tensor (asynchronous).  With gamma (float32 [K]) or c: of the gain-folded
    weight x[n, k] * RN_fp32(c * gamma[k]), x 2-D."""
    import torch
    if not (x.is_cuda and x.dtype == torch.bfloat16 and x.is_contiguous()):
        raise ValueError("x must be a contiguous bfloat16 CUDA tensor")
    out = _empty((1,), torch.float32, x.device, stream)
    if gamma is not None or c != 1.0:
        _check_gain(x, gamma)
        _launch(lib().mxnorm_absmax_gain_bf16, x.device, stream, x.data_ptr(), x.shape[0], x.shape[1], _ptr(gamma),
                float(c), out.data_ptr())
    else:
        _launch(lib().mxnorm_absmax_bf16, x.device, stream, x.data_ptr(), x.numel(), out.data_ptr())
    return out


def nvfp4_tensor_scale(x, stream=None):
    """The NVFP4 tensor scale of a contiguous bf16 CUDA tensor, derived by
    the library on the device (mxnorm_nvfp4_tensor_scale: the largest finite
    |x| / (448 * 6), rounded to fp32; 1 when there is none but zero).
    Returns a 1-element float32 CUDA tensor; asynchronous."""
    import torch
    if not (x.is_cuda and x.dtype == torch.bfloat16 and x.is_contiguous()):
        raise ValueError("x must be a contiguous bfloat16 CUDA tensor")
    out = _empty((1,), torch.float32, x.device, stream)
    _launch(lib().mxnorm_nvfp4_tensor_scale, x.device, stream, x.data_ptr(), x.numel(), out.data_ptr())
    return out


def quant_fwd_nvfp4(x, p: int = 2, tensor_scale=None, out=None, stream=None):
    """MXNorm over the NVFP4 cast of a contiguous bf16 CUDA tensor [..., H]
    (H % 16 == 0).  Returns (codes uint8 [..., H/2], scales uint8 [..., H/16]
    UE4M3, inv_rms float32 [...]).  tensor_scale: a float (passed by value),
    a 1-element float32 CUDA tensor (read by the kernel on the device), or
    None for nvfp4_tensor_scale(x) derived on the device (no host round
    trip either way but the float)."""
    import torch
    if not (x.is_cuda and x.dtype == torch.bfloat16 and x.is_contiguous()):
        raise ValueError("x must be a contiguous bfloat16 CUDA tensor")
    H = x.shape[-1]
    T = x.numel() // H if H else 0
    lead = tuple(x.shape[:-1])
    if tensor_scale is None:
        tensor_scale = nvfp4_tensor_scale(x, stream)
    if out is None:
        out = (_empty(lead + (H // 2,), torch.uint8, x.device, stream),
               _empty(lead + (H // 16,), torch.uint8, x.device, stream),
               _empty(lead, torch.float32, x.device, stream))
    codes, scales, inv = out
    _require(codes, "codes", x.device, min_numel=T * (H // 2), byte_elems=True)
    _require(scales, "scales", x.device, min_numel=T * (H // 16), byte_elems=True)
    _require(inv, "inv_rms", x.device, torch.float32, T)
    with _device(x.device):
        if isinstance(tensor_scale, torch.Tensor):
            _require(tensor_scale, "tensor_scale", x.device, torch.float32, 1)
            _check(lib().mxnorm_quant_fwd_nvfp4_dev(x.data_ptr(), T, H, int(p), tensor_scale.data_ptr(),
                                                    codes.data_ptr(), scales.data_ptr(), inv.data_ptr(),
                                                    _stream_ptr(x.device, stream)))
        else:
            _check(lib().mxnorm_quant_fwd_nvfp4(x.data_ptr(), T, H, int(p), float(tensor_scale), codes.data_ptr(),
                                                scales.data_ptr(), inv.data_ptr(), _stream_ptr(x.device, stream)))
    return codes, scales, inv


SCALE_LAYOUT = {"row_major": 0, "mma": 1}


def mma_scale_bytes(rows: int, H: int) -> int:
    """Bytes of an MMA-layout scale buffer for rows x H (H % 128 == 0)."""
    n = lib().mxnorm_mma_scale_bytes(rows, H)
    if n < 0:
        raise ValueError("the MMA scale layout needs H % 128 == 0")
    return n


def _scale_buffer(rows, H, layout, device, stream):
    import torch
    if layout == "mma":
        return _empty((mma_scale_bytes(rows, H),), torch.uint8, device, stream)
    return _empty((rows, H // 32), torch.uint8, device, stream)


def quant_fwd_mma(x, p: int = 2, fmt: str = "mxfp8", stream=None):
    """mxnorm_quant_fwd with the scales in the tensor-core MMA atom layout
    (for mxnorm_linear_fwd).  Returns (codes, scales (flat uint8), inv_rms)."""
    import torch
    if not (x.is_cuda and x.dtype == torch.bfloat16 and x.is_contiguous()):
        raise ValueError("x must be a contiguous bfloat16 CUDA tensor")
    H = x.shape[-1]
    T = x.numel() // H if H else 0
    codes = _empty(tuple(x.shape[:-1]) + (code_bytes(H, fmt),), torch.uint8, x.device, stream)
    scales = _scale_buffer(T, H, "mma", x.device, stream)
    inv = _empty(tuple(x.shape[:-1]), torch.float32, x.device, stream)
    with _device(x.device):
        _check(lib().mxnorm_quant_fwd_layout(x.data_ptr(), T, H, int(p), FMT[fmt], codes.data_ptr(),
                                             scales.data_ptr(), inv.data_ptr(), 1, _stream_ptr(x.device, stream)))
    return codes, scales, inv


def mx_cast(x, layout: str = "row_major", stream=None):
    """MXFP8 E4M3 cast alone (no estimator) of bf16 rows: (codes, scales)."""
    import torch
    if not (x.is_cuda and x.dtype == torch.bfloat16 and x.is_contiguous()):
        raise ValueError("x must be a contiguous bfloat16 CUDA tensor")
    H = x.shape[-1]
    T = x.numel() // H if H else 0
    codes = _empty(tuple(x.shape), torch.uint8, x.device, stream)
    scales = _scale_buffer(T, H, layout, x.device, stream)
    with _device(x.device):
        _check(lib().mx_cast_fwd(x.data_ptr(), T, H, 0, codes.data_ptr(), scales.data_ptr(), SCALE_LAYOUT[layout],
                                 _stream_ptr(x.device, stream)))
    return codes, scales


def mx_cast_gain(w, gamma, c: float = 1.0, layout: str = "mma", stream=None):
    """MXFP8 cast of MXNormLinear's gain-folded weight: rows of
    w[n, k] * RN_fp32(c * gamma[k]), each product rounded to fp32.
    w: contiguous bf16 CUDA tensor [N, K] (one row per output feature);
    gamma: contiguous float32 CUDA tensor [K].  Returns (codes, scales)."""
    import torch
    if not (w.is_cuda and w.dtype == torch.bfloat16 and w.is_contiguous() and w.dim() == 2):
        raise ValueError("w must be a contiguous 2-D bfloat16 CUDA tensor")
    N, K = w.shape
    _require(gamma, "gamma", w.device, torch.float32)
    if tuple(gamma.shape) != (K,):
        raise ValueError("gamma must hold K entries")
    codes = _empty((N, K), torch.uint8, w.device, stream)
    scales = _scale_buffer(N, K, layout, w.device, stream)
    with _device(w.device):
        _check(lib().mx_cast_gain_fwd(w.data_ptr(), N, K, gamma.data_ptr(), float(c), codes.data_ptr(),
                                      scales.data_ptr(), SCALE_LAYOUT[layout], _stream_ptr(w.device, stream)))
    return codes, scales


def linear_fwd(x_codes, x_scales, inv_rms, w_codes, w_scales, out=None, stream=None):
    """MXNormLinear's consumer GEMM on the tensor cores: out = bf16(inv_rms[t]
    * sum_k x^[t,k] w^[n,k]); scales in the MMA layout.  Returns out [T, N]."""
    import torch
    if getattr(x_codes, "dim", lambda: 0)() != 2 or getattr(w_codes, "dim", lambda: 0)() != 2:
        raise ValueError("x_codes and w_codes must be 2-D [rows, K]")
    T, K = x_codes.shape
    N = w_codes.shape[0]
    if w_codes.shape[1] != K:
        raise ValueError(f"w_codes has K = {w_codes.shape[1]}, x_codes has K = {K}")
    dev = x_codes.device
    _require(x_codes, "x_codes", dev, byte_elems=True)
    _require(w_codes, "w_codes", dev, byte_elems=True)
    if K % 128 == 0:  # else the C ABI reports the shape error
        _require(x_scales, "x_scales", dev, min_numel=mma_scale_bytes(T, K), byte_elems=True)
        _require(w_scales, "w_scales", dev, min_numel=mma_scale_bytes(N, K), byte_elems=True)
    _require(inv_rms, "inv_rms", dev, torch.float32, T)
    if out is None:
        out = _empty((T, N), torch.bfloat16, dev, stream)
    _require(out, "out", dev, torch.bfloat16, T * N)
    with _device(dev):
        _check(lib().mxnorm_linear_fwd(x_codes.data_ptr(), x_scales.data_ptr(), inv_rms.data_ptr(),
                                       w_codes.data_ptr(), w_scales.data_ptr(), T, K, N, out.data_ptr(),
                                       _stream_ptr(dev, stream)))
    return out


def bwd_ste(x, dy, inv_rms, out=None, stream=None):
    """Straight-through backward of MXNorm: dx = r dy - r^3 x mean(dy x)
    with r = inv_rms from the forward.  x, dy: contiguous bf16 CUDA tensors
    [..., H]; inv_rms: float32 [...].  Returns dx (bf16, like x)."""
    import torch
    for t in (x, dy):
        if not (t.is_cuda and t.dtype == torch.bfloat16 and t.is_contiguous()):
            raise ValueError("x and dy must be contiguous bfloat16 CUDA tensors")
    if dy.shape != x.shape or inv_rms.dtype != torch.float32 or not inv_rms.is_contiguous():
        raise ValueError("dy must match x, inv_rms must be contiguous float32")
    H = x.shape[-1]
    T = x.numel() // H if H else 0
    if inv_rms.numel() != T:
        raise ValueError("inv_rms needs one value per row")
    _require(dy, "dy", x.device)
    _require(inv_rms, "inv_rms", x.device, torch.float32, T)
    dx = _empty(tuple(x.shape), torch.bfloat16, x.device, stream) if out is None else out
    _require(dx, "out", x.device, torch.bfloat16, T * H)
    with _device(x.device):
        _check(lib().mxnorm_bwd_ste(x.data_ptr(), dy.data_ptr(), inv_rms.data_ptr(), T, H, dx.data_ptr(),
                                    _stream_ptr(x.device, stream)))
    return dx


# ------------------------------------------------------------ FP4 products
# Formats with 4-bit codes that linear_fwd_fp4 multiplies, and the ones
# mx_dequant reads back (FMT has the MX formats alone).
FP4_FMT = {"mxfp4": 1, "mxfp4_h16": 2, "mxfp4_h32": 4, "nvfp4": 6}
DEQUANT_FMT = {**FMT, "nvfp4": 6}


def _fmt_of(table, fmt):
    if fmt not in table:
        raise ValueError(f"fmt must be one of {', '.join(table)}, not {fmt!r}")
    return table[fmt]


def _layout_of(layout):
    if layout not in SCALE_LAYOUT:
        raise ValueError(f"layout must be one of {', '.join(SCALE_LAYOUT)}, not {layout!r}")
    return SCALE_LAYOUT[layout]


def _ptr(t):
    return None if t is None else t.data_ptr()


def _scale_bytes(rows, H, fmt, layout):
    """Bytes of the block scales of rows x H (mxnorm_mma_scale_bytes_fmt); 0
    for a length without the layout, which the C ABI reports."""
    blk = 16 if fmt == "nvfp4" else 32
    if layout != "mma":
        return rows * (H // blk)
    return 0 if H % (4 * blk) else (rows + 127) // 128 * (H // (4 * blk)) * 512


def _need_scales(t, name, index, rows, H, fmt, layout):
    """_need for block scales, and before it a refusal where their shape shows the
    other layout (row-major ones end in the row's blocks; the MMA layout is flat):
    either may be large enough for the other."""
    blocks = H // (16 if fmt == "nvfp4" else 32)
    dims = getattr(t, "shape", (blocks,))
    ends_in_blocks = len(dims) > 0 and dims[-1] == blocks
    if layout == "mma" and len(dims) > 1 and ends_in_blocks and rows > 1:
        raise ValueError(f"{name} has the row-major shape {tuple(dims)}: the MMA layout is flat")
    if layout != "mma" and not ends_in_blocks:
        raise ValueError(f"{name} must end in the row's {blocks} blocks in the row-major layout, not {tuple(dims)}")
    _need(t, name, index, _scale_bytes(rows, H, fmt, layout))


def _one_a_row(inv_rms, rows):
    if inv_rms.numel() != rows:
        raise ValueError(f"inv_rms holds {inv_rms.numel()} values for {rows} rows")


def _fp4_out(rows, K, fmt, layout, device, out, stream):
    """(codes [rows, K/2], scales) for a cast: the caller's, checked, or new ones."""
    import torch
    n = _scale_bytes(rows, K, fmt, layout)
    if out is None:
        shape = (n,) if layout == "mma" else (rows, K // (16 if fmt == "nvfp4" else 32))
        return (_empty((rows, K // 2), torch.uint8, device, stream), _empty(shape, torch.uint8, device, stream))
    codes, scales = out
    _need(codes, "codes", device.index, rows * (K // 2))
    _need(scales, "scales", device.index, n)
    return codes, scales


def _check_gain(w, gamma):
    import torch
    if not (w.is_cuda and w.dtype == torch.bfloat16 and w.is_contiguous() and w.dim() == 2):
        raise ValueError("w must be a contiguous 2-D bfloat16 CUDA tensor")
    if gamma is not None:
        _need(gamma, "gamma", w.get_device(), 0, torch.float32)
        if tuple(gamma.shape) != (w.shape[1],):
            raise ValueError("gamma must hold K entries")


def nvfp4_tensor_scale_gain(w, gamma=None, c: float = 1.0, stream=None):
    """The NVFP4 tensor scale of a gain-folded weight (the largest finite
    |w[n, k] * RN_fp32(c * gamma[k])| / (448 * 6); 1 where that is 0 in
    fp32), derived on the device.  Returns a 1-element float32 CUDA tensor."""
    import torch
    _check_gain(w, gamma)
    N, K = w.shape
    out = _empty((1,), torch.float32, w.device, stream)
    _launch(lib().mxnorm_nvfp4_tensor_scale_gain, w.device, stream, w.data_ptr(), N, K, _ptr(gamma), float(c),
            out.data_ptr())
    return out


def mx_cast_fp4(w, fmt: str = "mxfp4", gamma=None, c: float = 1.0, tensor_scale=None, layout: str = "mma", out=None,
                stream=None):
    """FP4 cast of a weight for linear_fwd_fp4: rows of w[n, k] * RN_fp32(c *
    gamma[k]) (gamma None: ones), rotated for "mxfp4_h16" / "mxfp4_h32",
    as E2M1 codes and block scales.  w: contiguous bf16 CUDA tensor [N, K].
    "nvfp4" takes the tensor scale as a 1-element float32 CUDA tensor, or
    derives it (nvfp4_tensor_scale_gain).  `out` may pass (codes, scales).
    Returns (codes uint8 [N, K/2], scales uint8, tensor_scale or None)."""
    import torch
    _check_gain(w, gamma)
    f, lay = _fmt_of(FP4_FMT, fmt), _layout_of(layout)
    N, K = w.shape
    codes, scales = _fp4_out(N, K, fmt, layout, w.device, out, stream)
    if fmt == "nvfp4":
        if tensor_scale is None:
            tensor_scale = nvfp4_tensor_scale_gain(w, gamma, c, stream)
        _need(tensor_scale, "tensor_scale", w.get_device(), 1, torch.float32)
    _launch(lib().mx_cast_fp4_fwd, w.device, stream, w.data_ptr(), N, K, f, _ptr(gamma), float(c),
            _ptr(tensor_scale), codes.data_ptr(), scales.data_ptr(), lay)
    return codes, scales, tensor_scale


def quant_fwd_nvfp4_mma(x, p: int = 2, tensor_scale=None, stream=None):
    """quant_fwd_nvfp4 with the scales in the tensor-core MMA atom layout (for
    linear_fwd_fp4; H % 64 == 0).  tensor_scale: a 1-element float32 CUDA
    tensor, or None to derive it on the device.  Returns (codes uint8
    [..., H/2], scales (flat uint8), inv_rms float32 [...], tensor_scale)."""
    import torch
    if not (x.is_cuda and x.dtype == torch.bfloat16 and x.is_contiguous()):
        raise ValueError("x must be a contiguous bfloat16 CUDA tensor")
    H = x.shape[-1]
    T = x.numel() // H if H else 0
    if tensor_scale is None:
        tensor_scale = nvfp4_tensor_scale(x, stream)
    _need(tensor_scale, "tensor_scale", x.get_device(), 1, torch.float32)
    codes = _empty(tuple(x.shape[:-1]) + (H // 2,), torch.uint8, x.device, stream)
    scales = _empty((_scale_bytes(T, H, "nvfp4", "mma"),), torch.uint8, x.device, stream)
    inv = _empty(tuple(x.shape[:-1]), torch.float32, x.device, stream)
    _launch(lib().mxnorm_quant_fwd_nvfp4_layout, x.device, stream, x.data_ptr(), T, H, int(p),
            tensor_scale.data_ptr(), codes.data_ptr(), scales.data_ptr(), inv.data_ptr(), 1)
    return codes, scales, inv, tensor_scale


def mx_dequant(codes, scales, fmt: str = "mxfp8", layout: str = "row_major", tensor_scale=None, out=None,
               stream=None):
    """The bf16 values that codes [..., H or H/2] and their block scales stand
    for.  Rotated formats give the rotated values: each aligned group of 16 or
    32 times the orthonormal Hadamard matrix in Sylvester order, its own
    inverse, so a gradient through a rotated weight, dout @ out, takes the
    matrix once more to leave the rotated basis.  Row-major scales end in the
    row's blocks, [..., H/32 or H/16]; the MMA layout is flat.  "nvfp4" takes the cast's
    tensor scale (1-element float32 CUDA tensor).  Returns bf16 [..., H]."""
    import torch
    f, lay = _fmt_of(DEQUANT_FMT, fmt), _layout_of(layout)
    dev = codes.device
    index = dev.index if dev.type == "cuda" else -2
    _need(codes, "codes", index, 0)
    per = 1 if fmt.startswith("mxfp8") else 2
    H = codes.shape[-1] * per
    T = codes.numel() * per // H if H else 0
    _need_scales(scales, "scales", index, T, H, fmt, layout)
    if tensor_scale is not None:
        _need(tensor_scale, "tensor_scale", index, 1, torch.float32)
    if out is None:
        out = _empty(tuple(codes.shape[:-1]) + (H,), torch.bfloat16, dev, stream)
    else:
        _need(out, "out", index, T * H, torch.bfloat16)
    _launch(lib().mx_dequant_fwd, dev, stream, codes.data_ptr(), scales.data_ptr(), T, H, f, lay, _ptr(tensor_scale),
            out.data_ptr())
    return out


def linear_fwd_fp4(x_codes, x_scales, inv_rms, w_codes, w_scales, fmt: str = "mxfp4", x_tensor_scale=None,
                   w_tensor_scale=None, out=None, stream=None, *, _drill=()):
    """MXNormLinear's product on FP4 codes: out = bf16(inv_rms[t] * g_x * g_w *
    sum_k x^[t, k] w^[n, k]) on the tensor cores; scales in the MMA layout.
    x_codes uint8 [T, K/2] (any T from a single token), w_codes uint8
    [N, K/2]; inv_rms float32 [T] or None (ones); the tensor scales are for
    "nvfp4".  Rows whose inv_rms is +Inf (NVFP4 rows without a value, such as
    padding) give zeros.  Returns out [T, N] (bf16)."""
    import torch
    f = _fmt_of(FP4_FMT, fmt)
    if getattr(x_codes, "dim", lambda: 0)() != 2 or getattr(w_codes, "dim", lambda: 0)() != 2:
        raise ValueError("x_codes and w_codes must be 2-D [rows, K/2]")
    T, K = x_codes.shape[0], 2 * x_codes.shape[1]
    N = w_codes.shape[0]
    if 2 * w_codes.shape[1] != K:
        raise ValueError(f"w_codes has K = {2 * w_codes.shape[1]}, x_codes has K = {K}")
    dev = x_codes.device
    index = dev.index if dev.type == "cuda" else -2
    _need(x_codes, "x_codes", index, 0)
    _need(w_codes, "w_codes", index, 0)
    _need_scales(x_scales, "x_scales", index, T, K, fmt, "mma")
    _need_scales(w_scales, "w_scales", index, N, K, fmt, "mma")
    if inv_rms is not None:
        _need(inv_rms, "inv_rms", index, T, torch.float32)
        _one_a_row(inv_rms, T)
    if x_tensor_scale is not None:
        _need(x_tensor_scale, "x_tensor_scale", index, 1, torch.float32)
    if w_tensor_scale is not None:
        _need(w_tensor_scale, "w_tensor_scale", index, 1, torch.float32)
    if out is None:
        out = _empty((T, N), torch.bfloat16, dev, stream)
    else:
        _need(out, "out", index, T * N, torch.bfloat16)
    fn = lib().mxnorm_linear_fp4_wait_drill if _drill else lib().mxnorm_linear_fp4_fwd
    _launch(fn, dev, stream, x_codes.data_ptr(), x_scales.data_ptr(), _ptr(inv_rms), w_codes.data_ptr(),
            w_scales.data_ptr(), T, K, N, f, _ptr(x_tensor_scale), _ptr(w_tensor_scale), out.data_ptr(), *_drill)
    return out


def linear_fp4_wait_drill(x_codes, x_scales, inv_rms, w_codes, w_scales, fmt: str = "mxfp4", x_tensor_scale=None,
                          w_tensor_scale=None, withheld_stage: int = 0, wait_limit_ns: int = 2_000_000, out=None,
                          stream=None):
    """Failure-detection drill (mxnorm_linear_fp4_wait_drill): the FP4 product
    with the loads of one stage withheld, so that its bounded waits expire
    and bit 3 of device_errors is set.  Returns out, whose values are invalid."""
    return linear_fwd_fp4(x_codes, x_scales, inv_rms, w_codes, w_scales, fmt, x_tensor_scale, w_tensor_scale, out,
                          stream, _drill=(int(withheld_stage), int(wait_limit_ns)))


# -------------------------------------------------------- 8-bit checkpoints
def bwd_ste_ckpt(x_codes, x_scales, dy, inv_rms, layout: str = "row_major", out=None, stream=None):
    """bwd_ste from the forward's MXFP8 codes and scales instead of its bf16
    input: dx = r dy - r^3 x^ mean(dy x^).  x_codes uint8 [..., H] and
    x_scales (in `layout`) as quant_fwd / quant_fwd_mma / mx_cast wrote them;
    dy: contiguous bf16 CUDA tensor like x; inv_rms float32 [...] (+Inf, a row
    without a value: its dx is 0).  Returns dx (bf16, like dy)."""
    import torch
    lay = _layout_of(layout)
    dev = dy.device
    index = dev.index if dev.type == "cuda" else -2
    _need(dy, "dy", index, 0, torch.bfloat16)
    shape = dy.shape
    if shape != x_codes.shape:
        raise ValueError("dy must match x_codes")
    H = shape[-1]
    T = dy.numel() // H if H else 0
    _need(x_codes, "x_codes", index, 0)
    _need_scales(x_scales, "x_scales", index, T, H, "mxfp8", layout)
    _need(inv_rms, "inv_rms", index, T, torch.float32)
    _one_a_row(inv_rms, T)
    if out is None:
        dx = _empty(shape, torch.bfloat16, dev, stream)
    else:
        dx = out
        _need(dx, "out", index, T * H, torch.bfloat16)
    _launch(lib().mxnorm_bwd_ste_ckpt, dev, stream, x_codes.data_ptr(), x_scales.data_ptr(), lay, dy.data_ptr(),
            inv_rms.data_ptr(), T, H, dx.data_ptr())
    return dx


def linear_wgrad_ckpt(x_codes, x_scales, inv_rms, dout, layout: str = "mma", out=None, stream=None, *, _drill=()):
    """Weight gradient of MXNormLinear from the MXFP8 checkpoint: dw[n, k] =
    bf16(sum_t dout[t, n] * RN_bf16(inv_rms[t] * x^[t, k])).  x_codes uint8
    [T, K] and x_scales (in `layout`) as the forward wrote them; inv_rms
    float32 [T] or None (ones; a row of +Inf adds nothing); dout: contiguous
    bf16 CUDA tensor [T, N] (N % 8 == 0).  A split sum's workspace is allocated
    per call (torch's allocator, on the call's stream).  Returns dw (bf16
    [N, K], overwritten)."""
    import torch
    lay = _layout_of(layout)
    if getattr(x_codes, "dim", lambda: 0)() != 2 or getattr(dout, "dim", lambda: 0)() != 2:
        raise ValueError("x_codes and dout must be 2-D [T, K] and [T, N]")
    T, K = x_codes.shape
    N = dout.shape[1]
    if dout.shape[0] != T:
        raise ValueError(f"dout has T = {dout.shape[0]}, x_codes has T = {T}")
    dev = x_codes.device
    index = dev.index if dev.type == "cuda" else -2
    _need(x_codes, "x_codes", index, 0)
    _need_scales(x_scales, "x_scales", index, T, K, "mxfp8", layout)
    _need(dout, "dout", index, 0, torch.bfloat16)
    if inv_rms is not None:
        _need(inv_rms, "inv_rms", index, T, torch.float32)
        _one_a_row(inv_rms, T)
    if out is None:
        dw = _empty((N, K), torch.bfloat16, dev, stream)
    else:
        dw = out
        _need(dw, "out", index, N * K, torch.bfloat16)
    need = lib().mxnorm_linear_wgrad_workspace_bytes(T, K, N)
    ws = _workspace((need,), torch.uint8, dev, stream) if need > 0 else None
    fn = lib().mxnorm_linear_wgrad_wait_drill if _drill else lib().mxnorm_linear_wgrad_ckpt
    _launch(fn, dev, stream, x_codes.data_ptr(), x_scales.data_ptr(), lay, _ptr(inv_rms), dout.data_ptr(),
            T, K, N, dw.data_ptr(), _ptr(ws), max(0, need), *_drill)
    return dw


def linear_wgrad_wait_drill(x_codes, x_scales, inv_rms, dout, layout: str = "mma", withheld_load: int = 0,
                            withheld_stage: int = 0, wait_limit_ns: int = 2_000_000, out=None, stream=None):
    """Failure-detection drill (mxnorm_linear_wgrad_wait_drill): the weight
    gradient with one load of its pipeline withheld (0: dout's, 1: the
    codes', of the given stage), so that its bounded waits expire and bit 4
    of device_errors is set.  Returns dw, whose values are invalid."""
    return linear_wgrad_ckpt(x_codes, x_scales, inv_rms, dout, layout, out, stream,
                             _drill=(int(withheld_load), int(withheld_stage), int(wait_limit_ns)))


def tiled_wait_drill(x, withheld_tile: int = 0, wait_limit_ns: int = 2_000_000, out=None, stream=None):
    """Failure-detection drill (mxnorm_tiled_wait_drill): the tiled MXFP8
    pass with one tile's copy withheld, so that its bounded waits expire
    after wait_limit_ns and bit 0 of device_errors() gets set.  Returns the
    (invalid) outputs (codes, scales, inv_rms)."""
    import torch
    if not (x.is_cuda and x.dtype == torch.bfloat16 and x.is_contiguous()):
        raise ValueError("x must be a contiguous bfloat16 CUDA tensor")
    H = x.shape[-1]
    T = x.numel() // H if H else 0
    if out is None:
        out = (_empty((T, H), torch.uint8, x.device, stream),
               _empty((T, H // 32), torch.uint8, x.device, stream),
               _empty((T,), torch.float32, x.device, stream))
    codes, scales, inv = out
    _require(codes, "codes", x.device, min_numel=T * H, byte_elems=True)
    _require(scales, "scales", x.device, min_numel=T * (H // 32), byte_elems=True)
    _require(inv, "inv_rms", x.device, torch.float32, T)
    with _device(x.device):
        _check(lib().mxnorm_tiled_wait_drill(x.data_ptr(), T, H, codes.data_ptr(), scales.data_ptr(),
                                             inv.data_ptr(), int(withheld_tile), int(wait_limit_ns),
                                             _stream_ptr(x.device, stream)))
    return codes, scales, inv


def device_errors(clear: bool = True) -> int:
    """The device error flags: bit 0, a bounded wait of the tiled kernel
    timed out; bit 1, a pipeline wait of the GEMM timed out; bit 2, a device
    NVFP4 tensor scale was not a finite positive float; bit 3, a pipeline
    wait of the FP4 product timed out; bit 4, one of the weight gradient."""
    v = ctypes.c_uint32(0)
    _check(lib().mxnorm_device_errors(ctypes.byref(v), int(clear)))
    return v.value


_host_ws = {}


def quant_fwd_host(x, p: int = 2, fmt: str = "mxfp8", out=None, device=None, chunks: int = 8,
                   variant: str = "auto", mode: str = "auto"):
    """MXNorm forward of a bf16 CPU tensor; returns (codes, scales, inv_rms)
    CPU tensors, valid once the current stream of `device` has synchronised.

    mode "zero_copy": x and the outputs are pinned host memory, which is
    mapped into the GPU's address space; the kernel reads x and writes its
    outputs across the host link directly (no staging buffers, no copy
    engine).  On Grace-Blackwell this runs at the host link's speed.
    mode "staged": the rows are split into `chunks` pieces over three CUDA
    streams: per piece a host->device copy of x, the C-ABI call, and
    device->host copies of codes, scales and inv_rms, so copies in both
    directions overlap with each other and with the kernels; device
    staging buffers are cached per (device, shape, fmt).
    mode "auto": zero_copy when x and every output are pinned, else staged.
    """
    import torch
    if x.is_cuda or x.dtype != torch.bfloat16 or not x.is_contiguous():
        raise ValueError("x must be a contiguous bfloat16 CPU tensor")
    device = torch.device(device if device is not None else "cuda")
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    H = x.shape[-1]
    T = x.numel() // H if H else 0
    cb = code_bytes(H, fmt)
    if out is None:
        out = (torch.empty((T, cb), dtype=torch.uint8).pin_memory(),
               torch.empty((T, H // 32), dtype=torch.uint8).pin_memory(),
               torch.empty((T,), dtype=torch.float32).pin_memory())
    pinned = x.is_pinned() and all(t.is_pinned() and t.is_contiguous() for t in out)
    if mode == "auto":
        mode = "zero_copy" if pinned else "staged"
    if mode == "zero_copy":
        if not pinned:
            raise ValueError("zero_copy needs x and every output in pinned (page-locked) host memory")
        with _device(device):
            _check(lib().mxnorm_quant_fwd_ex(x.data_ptr(), T, H, int(p), FMT[fmt], out[0].data_ptr(),
                                             out[1].data_ptr(), out[2].data_ptr(), VARIANT[variant],
                                             _stream_ptr(device, None)))
        return out
    if mode != "staged":
        raise ValueError(f"unknown mode {mode!r}")
    oc, os_, oi = (t.view(-1) for t in out)
    key = (device.index, T, H, fmt)
    ws = _host_ws.get(key)
    if ws is None:
        ws = {"x": torch.empty((T, H), dtype=torch.bfloat16, device=device),
              "c": torch.empty((T, cb), dtype=torch.uint8, device=device),
              "s": torch.empty((T, H // 32), dtype=torch.uint8, device=device),
              "i": torch.empty((T,), dtype=torch.float32, device=device),
              "streams": [torch.cuda.Stream(device=device) for _ in range(3)]}
        _host_ws[key] = ws
    xv = x.view(T, H)
    cur = torch.cuda.current_stream(device)
    streams = ws["streams"]
    for s in streams:
        s.wait_stream(cur)
    rc = max(1, -(-T // max(1, chunks)))
    L = lib()
    for j, r0 in enumerate(range(0, T, rc)):
        r1 = min(T, r0 + rc)
        s = streams[j % len(streams)]
        with torch.cuda.stream(s):
            xd = ws["x"][r0:r1]
            xd.copy_(xv[r0:r1], non_blocking=True)
            cd, sd, idd = ws["c"][r0:r1], ws["s"][r0:r1], ws["i"][r0:r1]
            _check(L.mxnorm_quant_fwd_ex(xd.data_ptr(), r1 - r0, H, int(p), FMT[fmt], cd.data_ptr(),
                                         sd.data_ptr(), idd.data_ptr(), VARIANT[variant],
                                         ctypes.c_void_p(s.cuda_stream)))
            oc[r0 * cb:r1 * cb].copy_(cd.reshape(-1), non_blocking=True)
            os_[r0 * (H // 32):r1 * (H // 32)].copy_(sd.reshape(-1), non_blocking=True)
            oi[r0:r1].copy_(idd, non_blocking=True)
    for s in streams:
        cur.wait_stream(s)
    return out
