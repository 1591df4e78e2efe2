"""The root-mean-square norm before a projection, and 8-bit codes of rows
(argument marshalling; the work is proj_rms_norm and proj_quant_rows).

On the vLLM API page "vllm.models.kimi_k3.nvidia.specialized_decode.runtime.
hybrid" (section "HybridStep.run") every layer of a decode step adds the
residual and normalises the rows before its input projection and before its
MoE layer; the codes feed the 8-bit projection (PlanI8).
"""
from __future__ import annotations

import torch

from ._binding import _check, _lib, _on_current_device, _stream_handle

_BF16, _FP32 = torch.bfloat16, torch.float32


def _rows(x):
    """(rows, D, row stride) of BF16 rows."""
    if x.dtype is not _BF16:
        raise TypeError("x must be bfloat16")
    shape = x.shape
    if len(shape) != 2:
        raise ValueError("x must be [rows, D]")
    rows, D = shape
    ldx, one = x.stride()
    if one != 1 and rows > 0:
        raise ValueError("x must have unit column stride")
    if rows > 1 and ldx < D:
        raise ValueError("the rows of x overlap")
    return rows, D, ldx if rows > 1 else D


def _like(t, shape, dtype, name):
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of shape {tuple(shape)}")


def _norm(x, weight, residual, eps, out, codes, scale, stream):
    rows, D, ldx = _rows(x)
    if weight.dtype is not _BF16:
        raise TypeError("weight must be bfloat16")
    if weight.shape != (D,) or not weight.is_contiguous():
        raise ValueError(f"weight must be a contiguous tensor of shape ({D},)")
    tensors = [x, weight]
    rp, ldr, wide = None, D, 0
    if residual is not None:
        wide = residual.dtype is _FP32
        if not wide and residual.dtype is not _BF16:
            raise TypeError("residual must be bfloat16 or float32")
        if residual.shape != x.shape or (residual.stride(1) != 1 and rows > 0):
            raise ValueError("residual must have the shape of x and unit column stride")
        if rows > 1:
            ldr = residual.stride(0)
            if ldr < D:
                raise ValueError("the rows of residual overlap")
        rp = residual.data_ptr()
        tensors.append(residual)
    yp = cp = sp = None
    if out is not None:
        yp = out.data_ptr()
        tensors.append(out)
    if codes is not None:
        cp, sp = codes.data_ptr(), scale.data_ptr()
        tensors += (codes, scale)
    _on_current_device(*tensors)
    rc = _lib().proj_rms_norm(rows, D, x.data_ptr(), ldx, rp, ldr, wide, weight.data_ptr(), eps,
                              yp, cp, sp, _stream_handle(stream))
    if rc:
        _check(rc, f"proj_rms_norm(rows={rows}, D={D})")


def rms_norm(x, weight, *, residual=None, eps: float = 1e-6, out=None, stream=None):
    """BF16 rows (x + residual) * weight / rms(x + residual); the residual
    (bfloat16 or float32) is updated in place to the sum.  Returns `out`."""
    if out is None:
        out = x.new_empty(x.shape)
    else:
        _like(out, x.shape, _BF16, "out")
    _norm(x, weight, residual, eps, out, None, None, stream)
    return out


def _codes_of(x, codes, scale):
    if codes is None:
        codes = x.new_empty(x.shape, dtype=torch.int8)
    else:
        _like(codes, x.shape, torch.int8, "codes")
    if scale is None:
        scale = x.new_empty(x.shape[:1], dtype=_FP32)
    else:
        _like(scale, x.shape[:1], _FP32, "scale")
    return codes, scale


def rms_norm_i8(x, weight, *, residual=None, eps: float = 1e-6, codes=None, scale=None, out=None,
                stream=None):
    """As rms_norm, with the result in 8 bits: returns (codes, scale), int8
    [rows, D] and float32 [rows], standing for codes * scale.  With `out` the
    BF16 rows are written too."""
    codes, scale = _codes_of(x, codes, scale)
    if out is not None:
        _like(out, x.shape, _BF16, "out")
    _norm(x, weight, residual, eps, out, codes, scale, stream)
    return codes, scale


def quant_rows(x, *, codes=None, scale=None, stream=None):
    """8-bit codes of BF16 rows with a scale each, (codes, scale): activations
    take a scale per token, a weight [N, K] one per output channel."""
    rows, D, ldx = _rows(x)
    codes, scale = _codes_of(x, codes, scale)
    _on_current_device(x, codes, scale)
    rc = _lib().proj_quant_rows(rows, D, x.data_ptr(), ldx, codes.data_ptr(), scale.data_ptr(),
                                _stream_handle(stream))
    if rc:
        _check(rc, f"proj_quant_rows(rows={rows}, D={D})")
    return codes, scale
