"""Thin ctypes binding of the microscaled 4-bit operators of liblnq.so, with the entry-point names
of include/lnq_fp4.h.

Argument marshalling only, as in binding.py: PyTorch supplies device memory and the stream. Unlike
the entry points there, these take matrices whose rows are strided, and run on the device that
holds their tensors whichever device is current.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from .binding import LnqError, lib as _library

LNQ_FP4_MX, LNQ_FP4_NV = 0, 1
_DTYPE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
MAX_EXPERTS = 1024

EXPORTED = ("lnq_fp4_code_bytes", "lnq_fp4_scale_bytes", "lnq_fp4_tensor_scale",
            "lnq_fp4_quantize", "lnq_fp4_dequantize", "lnq_fp4_gemv", "lnq_fp4_grouped_gemv",
            "lnq_fp4_gemm", "lnq_fp4_grouped_gemm", "lnq_fp4_check")

_VP, _I64, _INT = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
_lib = None
_entry = {}  # name -> entry point, once loaded


def lib():
    """The loaded library with these entry points' signatures (raises if it was not built)."""
    global _lib
    if _lib is None:
        L = _library()
        L.lnq_fp4_code_bytes.argtypes, L.lnq_fp4_code_bytes.restype = [_I64], _I64
        L.lnq_fp4_scale_bytes.argtypes, L.lnq_fp4_scale_bytes.restype = [_I64, _INT], _I64
        L.lnq_fp4_tensor_scale.argtypes = [_VP, _INT, _I64, _I64, _I64, _VP, _VP]
        L.lnq_fp4_quantize.argtypes = [_VP, _INT, _I64, _I64, _I64, _INT, _VP, _VP, _VP, _VP]
        L.lnq_fp4_dequantize.argtypes = [_VP, _VP, _I64, _I64, _INT, _VP, _VP, _INT, _I64, _VP]
        L.lnq_fp4_gemv.argtypes = [_VP, _INT, _I64, _I64, _VP, _VP, _VP, _I64, _I64, _INT, _VP,
                                   _INT, _I64, _VP]
        L.lnq_fp4_grouped_gemv.argtypes = [_VP, _INT, _I64, _I64, _VP, _I64, _VP, _VP, _VP, _I64,
                                           _I64, _INT, _VP, _INT, _I64, _VP]
        L.lnq_fp4_gemm.argtypes = [_VP, _VP, _VP, _I64, _VP, _VP, _VP, _I64, _I64, _INT, _VP, _INT,
                                   _I64, _VP]
        L.lnq_fp4_grouped_gemm.argtypes = [_VP, _VP, _VP, _I64, _VP, _I64, _VP, _VP, _VP, _I64,
                                           _I64, _INT, _VP, _INT, _I64, _VP]
        L.lnq_fp4_check.argtypes = [_VP]
        for name in EXPORTED[2:]:
            getattr(L, name).restype = _INT
            _entry[name] = getattr(L, name)
        _lib = L
    return _lib


def lnq_fp4_code_bytes(d: int) -> int:
    """Bytes per row of codes (see include/lnq_fp4.h)."""
    return int(lib().lnq_fp4_code_bytes(int(d)))


def lnq_fp4_scale_bytes(d: int, fmt: int) -> int:
    """Bytes per row of scales (see include/lnq_fp4.h)."""
    return int(lib().lnq_fp4_scale_bytes(int(d), int(fmt)))


def _need(t, dtype, shape, name, device):
    """A contiguous CUDA tensor of this type and shape, on `device`."""
    if t.dtype != dtype or t.shape != shape or t.device != device or not t.is_cuda \
            or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous CUDA {dtype} {tuple(shape)} on {device}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")


def _dense(t, name, shape=None, device=None) -> Tuple[int, int]:
    """(type selector, row pitch) of an unquantised matrix [rows][d]; its rows may be strided."""
    kind, got = _DTYPE.get(t.dtype), t.shape
    if (kind is None or len(got) != 2 or got[1] < 1 or not t.is_cuda
            or (shape is not None and (got != shape or t.device != device))):
        raise ValueError(f"{name}: expected a CUDA float32, bfloat16 or float16 matrix"
                         f"{'' if shape is None else f' {tuple(shape)} on {device}'}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")
    rows, d = got
    if t.is_contiguous():
        return kind, d
    pitch, step = t.stride()
    pitch = pitch if rows > 1 else d
    if pitch < d or (d > 1 and step != 1):
        raise ValueError(f"{name}: expected rows of consecutive elements that do not overlap, got "
                         f"strides {t.stride()}")
    return kind, pitch


def _format(fmt) -> int:
    if fmt != LNQ_FP4_MX and fmt != LNQ_FP4_NV:
        raise ValueError(f"fmt: expected LNQ_FP4_MX or LNQ_FP4_NV, got {fmt!r}")
    return int(fmt)


def _out_type(dtype):
    if dtype not in _DTYPE:
        raise ValueError(f"dtype: expected float32, bfloat16 or float16, got {dtype}")
    return dtype


def _pitches(d, fmt) -> Tuple[int, int]:
    """Bytes per row of codes and of scales."""
    pad = -(-d // 128)
    return pad * 64, pad * (4 if fmt == LNQ_FP4_MX else 8)


def _codes(codes, scales, d, fmt, names, device, lead):
    """Checks the stored form of matrices [*lead][d]."""
    of_codes, of_scales = _pitches(d, fmt)
    _need(codes, torch.uint8, (*lead, of_codes), names[0], device)
    _need(scales, torch.uint8, (*lead, of_scales), names[1], device)


_INPUT, _WEIGHT = ("codes", "scales"), ("weight codes", "weight scales")
_ACTIVATION = ("activation codes", "activation scales")


def _scale(t, count, fmt, name, device):
    """The pointer of `count` matrix scales; MX has none."""
    if t is None:
        return None
    if fmt == LNQ_FP4_MX:
        raise ValueError(f"{name}: LNQ_FP4_MX has no matrix scale")
    if t.dtype != torch.float32 or t.numel() != count or t.device != device \
            or not t.is_contiguous():
        raise ValueError(f"{name}: expected {count} contiguous CUDA float32 on {device}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _empty(like, shape, dtype, stream):
    """An uninitialised tensor on the device of `like`, from the memory of the stream that the call
    runs on (as in binding.py)."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _output(y, like, shape, dtype, stream):
    """(y, its type selector, its row pitch): the y given, or a new one of `dtype`."""
    if y is None:
        return _empty(like, shape, _out_type(dtype), stream), _DTYPE[dtype], shape[1]
    return y, *_dense(y, "y", shape, like.device)


def _call(name, device, stream, *args):
    """Calls the entry point with the tensors' device current, on `stream` or that device's
    current stream."""
    index = device.index
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(index)
    elif stream.device != device:
        raise ValueError(f"{name}: the stream is of {stream.device}, the tensors are on {device}")
    else:
        handle = stream.cuda_stream
    entry = _entry.get(name) or getattr(lib(), name)
    if torch._C._cuda_getDevice() == index:
        status = entry(*args, handle)
    else:
        with torch.cuda.device(index):
            status = entry(*args, handle)
    if status:
        raise LnqError(status, name)


def lnq_fp4_tensor_scale(x: torch.Tensor, t: Optional[torch.Tensor] = None,
                         stream=None) -> torch.Tensor:
    """t [1]: the matrix scale of LNQ_FP4_NV for x [rows][d], the largest finite |x| / 2688."""
    xt, ldx = _dense(x, "x")
    if t is None:
        t = _empty(x, (1,), torch.float32, stream)
    _need(t, torch.float32, (1,), "t", x.device)
    _call("lnq_fp4_tensor_scale", x.device, stream, x.data_ptr(), xt, x.shape[0], x.shape[1], ldx,
          t.data_ptr())
    return t


def lnq_fp4_quantize(x: torch.Tensor, fmt: int, tensor_scale: Optional[torch.Tensor] = None,
                     codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                     stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """x [rows][d] -> (codes, scales), uint8 [rows][lnq_fp4_code_bytes(d)] and
    [rows][lnq_fp4_scale_bytes(d, fmt)]."""
    xt, ldx = _dense(x, "x")
    fmt, (rows, d), dev = _format(fmt), x.shape, x.device
    ts = _scale(tensor_scale, 1, fmt, "tensor_scale", dev)
    of_codes, of_scales = _pitches(d, fmt)
    if codes is None:
        codes = _empty(x, (rows, of_codes), torch.uint8, stream)
    else:
        _need(codes, torch.uint8, (rows, of_codes), "codes", dev)
    if scales is None:
        scales = _empty(x, (rows, of_scales), torch.uint8, stream)
    else:
        _need(scales, torch.uint8, (rows, of_scales), "scales", dev)
    _call("lnq_fp4_quantize", dev, stream, x.data_ptr(), xt, rows, d, ldx, fmt, ts,
          codes.data_ptr(), scales.data_ptr())
    return codes, scales


def lnq_fp4_dequantize(codes: torch.Tensor, scales: torch.Tensor, d: int, fmt: int,
                       tensor_scale: Optional[torch.Tensor] = None,
                       dtype: torch.dtype = torch.float32, y: Optional[torch.Tensor] = None,
                       stream=None) -> torch.Tensor:
    """The values [rows][d] that (codes, scales) stand for; `dtype` is y's where y is given."""
    fmt, d, dev = _format(fmt), int(d), codes.device
    rows = codes.shape[0]
    _codes(codes, scales, d, fmt, _INPUT, dev, (rows,))
    ts = _scale(tensor_scale, 1, fmt, "tensor_scale", dev)
    y, yt, ldy = _output(y, codes, (rows, d), dtype, stream)
    _call("lnq_fp4_dequantize", dev, stream, codes.data_ptr(), scales.data_ptr(), rows, d, fmt, ts,
          y.data_ptr(), yt, ldy)
    return y


def _offsets(offsets, experts, device):
    if not 1 <= experts <= MAX_EXPERTS:
        raise ValueError(f"experts: expected 1 .. {MAX_EXPERTS}, got {experts}")
    _need(offsets, torch.int32, (experts + 1,), "offsets", device)


def _gemv(name, x, offsets, codes, scales, fmt, tensor_scale, y, dtype, stream):
    xt, ldx = _dense(x, "x")
    fmt, (n, d_in), dev = _format(fmt), x.shape, x.device
    lead = codes.shape[:-1]
    grouped = offsets is not None
    if len(lead) != 1 + grouped:
        raise ValueError(f"codes: expected {'[experts][d_out][bytes]' if grouped else '[d_out][bytes]'}"
                         f", got {tuple(codes.shape)}")
    _codes(codes, scales, d_in, fmt, _WEIGHT, dev, lead)
    ts = _scale(tensor_scale, lead[0] if grouped else 1, fmt, "tensor_scale", dev)
    if grouped:
        _offsets(offsets, lead[0], dev)
    y, yt, ldy = _output(y, codes, (n, lead[-1]), dtype or x.dtype, stream)
    group = (offsets.data_ptr(), lead[0]) if grouped else ()
    _call(name, dev, stream, x.data_ptr(), xt, n, ldx, *group, codes.data_ptr(),
          scales.data_ptr(), ts, lead[-1], d_in, fmt, y.data_ptr(), yt, ldy)
    return y


def lnq_fp4_gemv(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, fmt: int,
                 tensor_scale: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                 dtype: Optional[torch.dtype] = None, stream=None) -> torch.Tensor:
    """y [nb][d_out] = x [nb][d_in] times the quantised matrix [d_out][d_in]. y's type is x's, or
    `dtype`, or that of the y given."""
    return _gemv("lnq_fp4_gemv", x, None, codes, scales, fmt, tensor_scale, y, dtype, stream)


def lnq_fp4_grouped_gemv(x: torch.Tensor, offsets: torch.Tensor, codes: torch.Tensor,
                         scales: torch.Tensor, fmt: int,
                         tensor_scale: Optional[torch.Tensor] = None,
                         y: Optional[torch.Tensor] = None, dtype: Optional[torch.dtype] = None,
                         stream=None) -> torch.Tensor:
    """lnq_fp4_gemv with the rows offsets[e] .. offsets[e+1] - 1 of x (int32 [experts + 1]) times
    matrix e of codes [experts][d_out][...]. Rows outside every group are left as they were."""
    return _gemv("lnq_fp4_grouped_gemv", x, offsets, codes, scales, fmt, tensor_scale, y, dtype,
                 stream)


def _gemm(name, a_codes, a_scales, offsets, codes, scales, d_in, fmt, a_scale, b_scale, dtype, y,
          stream):
    fmt, d_in, dev = _format(fmt), int(d_in), a_codes.device
    if d_in < 1:
        raise ValueError(f"d_in: expected at least 1, got {d_in}")
    n = a_codes.shape[0]
    lead = codes.shape[:-1]
    grouped = offsets is not None
    if len(lead) != 1 + grouped:
        raise ValueError(f"codes: expected {'[experts][d_out][bytes]' if grouped else '[d_out][bytes]'}"
                         f", got {tuple(codes.shape)}")
    _codes(a_codes, a_scales, d_in, fmt, _ACTIVATION, dev, (n,))
    _codes(codes, scales, d_in, fmt, _WEIGHT, dev, lead)
    ta = _scale(a_scale, 1, fmt, "a_scale", dev)
    tb = _scale(b_scale, lead[0] if grouped else 1, fmt, "b_scale", dev)
    if grouped:
        _offsets(offsets, lead[0], dev)
    y, yt, ldy = _output(y, codes, (n, lead[-1]), dtype, stream)
    group = (offsets.data_ptr(), lead[0]) if grouped else ()
    _call(name, dev, stream, a_codes.data_ptr(), a_scales.data_ptr(), ta, n, *group,
          codes.data_ptr(), scales.data_ptr(), tb, lead[-1], d_in, fmt, y.data_ptr(), yt, ldy)
    return y


def lnq_fp4_gemm(a_codes: torch.Tensor, a_scales: torch.Tensor, b_codes: torch.Tensor,
                 b_scales: torch.Tensor, d_in: int, fmt: int,
                 a_scale: Optional[torch.Tensor] = None, b_scale: Optional[torch.Tensor] = None,
                 dtype: torch.dtype = torch.bfloat16, y: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """y [n][d_out]: quantised activations [n][d_in] times the quantised matrix [d_out][d_in];
    a_scale and b_scale are their matrix scales."""
    return _gemm("lnq_fp4_gemm", a_codes, a_scales, None, b_codes, b_scales, d_in, fmt, a_scale,
                 b_scale, dtype, y, stream)


def lnq_fp4_grouped_gemm(a_codes: torch.Tensor, a_scales: torch.Tensor, offsets: torch.Tensor,
                         b_codes: torch.Tensor, b_scales: torch.Tensor, d_in: int, fmt: int,
                         a_scale: Optional[torch.Tensor] = None,
                         b_scale: Optional[torch.Tensor] = None,
                         dtype: torch.dtype = torch.bfloat16, y: Optional[torch.Tensor] = None,
                         stream=None) -> torch.Tensor:
    """lnq_fp4_gemm with the rows offsets[e] .. offsets[e+1] - 1 of the activations (int32
    [experts + 1]) times matrix e of b_codes [experts][d_out][...]; b_scale is [experts]. Rows
    outside every group are left as they were."""
    return _gemm("lnq_fp4_grouped_gemm", a_codes, a_scales, offsets, b_codes, b_scales, d_in, fmt,
                 a_scale, b_scale, dtype, y, stream)


def lnq_fp4_check(device=None, stream=None) -> int:
    """Synchronises the stream (the current one by default) and returns LNQ_OK, or LNQ_ERR_TIMEOUT
    if a product on it, or for the default stream any product of `device` (the stream's or the
    current one by default), has given up since its last report (see include/lnq_fp4.h)."""
    if device is None and stream is not None:
        device = stream.device
    with torch.cuda.device(device):
        if stream is None:
            stream = torch.cuda.current_stream()
        return int(lib().lnq_fp4_check(stream.cuda_stream))
