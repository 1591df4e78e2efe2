"""The root-mean-square norm before a projection, and 8-bit codes of rows
(argument marshalling; the work is proj_rms_norm and proj_quant_rows).

On the vLLM API page "vllm.models.kimi_k3.nvidia.specialized_decode.runtime.
hybrid" (section "HybridStep.run") every layer of a decode step adds the
residual and normalises the rows before its input projection and before its
MoE layer; the codes feed the 8-bit projection (PlanI8).
"""
from __future__ import annotations

from ._binding import _check, _lib, _on_current_device, _stream_handle


def _rows(x, name="x"):
    import torch
    if x.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16")
    if x.dim() != 2 or (x.shape[0] > 0 and x.stride(1) != 1):
        raise ValueError(f"{name} must be [rows, D] with unit column stride")
    return x.shape[0], x.shape[1], x.stride(0) if x.shape[0] > 1 else x.shape[1]


def _out(t, shape, dtype, like, name):
    import torch
    if t is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of shape {shape}")
    return t


def _norm(x, weight, residual, eps, y, codes, scale, stream):
    import torch
    rows, D, ldx = _rows(x)
    if weight.dtype != torch.bfloat16:
        raise TypeError("weight must be bfloat16")
    if tuple(weight.shape) != (D,) or not weight.is_contiguous():
        raise ValueError(f"weight must be a contiguous tensor of shape ({D},)")
    ops = [t for t in (x, weight, residual, y, codes, scale) if t is not None]
    _on_current_device(*ops)
    rp, ldr, wide = None, D, 0
    if residual is not None:
        if residual.dtype not in (torch.bfloat16, torch.float32):
            raise TypeError("residual must be bfloat16 or float32")
        if residual.shape != x.shape or (rows > 0 and residual.stride(1) != 1):
            raise ValueError("residual must have the shape of x and unit column stride")
        rp, wide = residual.data_ptr(), int(residual.dtype == torch.float32)
        ldr = residual.stride(0) if rows > 1 else D
    rc = _lib().proj_rms_norm(
        rows, D, x.data_ptr(), ldx, rp, ldr, wide, weight.data_ptr(), eps,
        None if y is None else y.data_ptr(), None if codes is None else codes.data_ptr(),
        None if scale is None else scale.data_ptr(), _stream_handle(stream))
    if rc:
        _check(rc, f"proj_rms_norm(rows={rows}, D={D})")


def rms_norm(x, weight, *, residual=None, eps: float = 1e-6, out=None, stream=None):
    """BF16 rows (x + residual) * weight / rms(x + residual); the residual
    (bfloat16 or float32) is updated in place to the sum.  Returns `out`."""
    import torch
    out = _out(out, tuple(x.shape), torch.bfloat16, x, "out")
    _norm(x, weight, residual, eps, out, None, None, stream)
    return out


def rms_norm_i8(x, weight, *, residual=None, eps: float = 1e-6, codes=None, scale=None, out=None,
                stream=None):
    """As rms_norm, with the result in 8 bits: returns (codes, scale), int8
    [rows, D] and float32 [rows], standing for codes * scale.  With `out` the
    BF16 rows are written too."""
    import torch
    shape = tuple(x.shape)
    codes = _out(codes, shape, torch.int8, x, "codes")
    scale = _out(scale, shape[:1], torch.float32, x, "scale")
    if out is not None:
        _out(out, shape, torch.bfloat16, x, "out")
    _norm(x, weight, residual, eps, out, codes, scale, stream)
    return codes, scale


def quant_rows(x, *, codes=None, scale=None, stream=None):
    """8-bit codes of BF16 rows with a scale each, (codes, scale): activations
    take a scale per token, a weight [N, K] one per output channel."""
    import torch
    rows, D, ldx = _rows(x)
    codes = _out(codes, (rows, D), torch.int8, x, "codes")
    scale = _out(scale, (rows,), torch.float32, x, "scale")
    _on_current_device(x, codes, scale)
    rc = _lib().proj_quant_rows(rows, D, x.data_ptr(), ldx, codes.data_ptr(), scale.data_ptr(),
                                _stream_handle(stream))
    if rc:
        _check(rc, f"proj_quant_rows(rows={rows}, D={D})")
    return codes, scale
