"""The gated delta rule between a KDA layer's two projections (argument
marshalling; the work is proj_delta_step and proj_delta_run).

On the vLLM API page "vllm.models.kimi_k3.nvidia.specialized_decode.runtime.
dep" (section "DepKda") the core between the packed input projection and
o_proj is a recurrence over a state per request, for single tokens and for
verify steps of several; delta_step is that recurrence and DeltaPlan its
chunked form for prompts.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from ._binding import (PLAN_HOST_ONLY, DeltaIO, _check, _lib, _on_current_device, _same_device,
                       _stream_handle)

HEAD = 128
_BF16, _FP32 = torch.bfloat16, torch.float32
# DeltaIO as bytes, in half the time a ctypes structure takes to fill
_IO = struct.Struct("5P5l4Plfii4x")
assert _IO.size == ctypes.sizeof(DeltaIO)


def _heads(t, name):
    """(rows, heads, row stride) of BF16 [rows, heads, 128]."""
    if t.dtype is not _BF16:
        raise TypeError(f"{name} must be bfloat16")
    shape = t.shape              # every attribute of a tensor is a call: each once
    if len(shape) != 3 or shape[2] != HEAD:
        raise ValueError(f"{name} must be [rows, heads, {HEAD}]")
    rows, h, _ = shape
    ld, lh, one = t.stride()
    if rows > 0 and (one != 1 or (h > 1 and lh != HEAD)):
        raise ValueError(f"the heads of a row of {name} must be contiguous")
    if rows <= 1:
        return rows, h, h * HEAD
    if ld < h * HEAD:
        raise ValueError(f"the rows of {name} overlap")
    return rows, h, ld


def _flat(t, rows, h, name):
    """Row stride of BF16 [rows, heads]."""
    if t.shape != (rows, h):
        raise ValueError(f"{name} must be [rows, heads]" +
                         (" or [rows, heads, 128]" if name == "f" else ""))
    ld, one = t.stride()
    if rows > 0 and h > 1 and one != 1:
        raise ValueError(f"{name} must have unit column stride")
    if rows > 1 and ld < h:
        raise ValueError(f"the rows of {name} overlap")
    return ld if rows > 1 else h


def _operands(q, k, v, f, b, a_log, dt_bias, state, out, scale, l2norm):
    """Checks what both forms take; returns (io, out, rows, heads, qk_heads, slots)."""
    rows, Hk, ldq = _heads(q, "q")
    rk, hk, ldk = _heads(k, "k")
    rv, H, ldv = _heads(v, "v")
    if rk != rows or hk != Hk or rv != rows or Hk < 1 or H % Hk:
        raise ValueError("q and k must have one shape, and v the same rows and a multiple of "
                         "their heads")
    if f.dtype is not _BF16 or b.dtype is not _BF16:
        raise TypeError("f and b must be bfloat16")
    head_gate = f.dim() == 2
    if head_gate:
        ldf, gates = _flat(f, rows, H, "f"), (H,)
    else:
        rf, hf, ldf = _heads(f, "f")
        if rf != rows or hf != H:
            raise ValueError("f must be [rows, heads] or [rows, heads, 128]")
        gates = (H, HEAD)
    ldb = _flat(b, rows, H, "b")
    if a_log.dtype is not _FP32 or dt_bias.dtype is not _FP32 or state.dtype is not _FP32:
        raise TypeError("a_log, dt_bias and state must be float32")
    if a_log.shape != (H,) or dt_bias.shape != gates or \
            not (a_log.is_contiguous() and dt_bias.is_contiguous()):
        raise ValueError(f"a_log must be [{H}] and dt_bias {list(gates)}, contiguous")
    shape = state.shape
    pool = shape[0]
    if shape != (pool, H, HEAD, HEAD) or pool < 1 or not state.is_contiguous():
        raise ValueError(f"state must be contiguous [slots, {H}, {HEAD}, {HEAD}]")
    if out is None:
        out = v.new_empty((rows, H, HEAD))
        ldo = H * HEAD
    else:
        ro, ho, ldo = _heads(out, "out")
        if ro != rows or ho != H:
            raise ValueError("out must have the shape of v")
    io = _IO.pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), f.data_ptr(), b.data_ptr(), ldq, ldk,
                  ldv, ldf, ldb, a_log.data_ptr(), dt_bias.data_ptr(), state.data_ptr(),
                  out.data_ptr(), ldo, HEAD ** -0.5 if scale is None else scale, bool(l2norm),
                  head_gate)
    return io, out, rows, H, Hk, pool


def delta_step(q, k, v, f, b, a_log, dt_bias, state, slots, *, tokens: int = 1, scale=None,
               l2norm: bool = True, out=None, stream=None):
    """The recurrent form: request i has rows [i * tokens, (i + 1) * tokens)
    and continues state[slots[i]] (int32 on the device; -1 is padding, whose
    rows of out become zero).  Updates state in place and returns out.

    q, k: bfloat16 [rows, qk_heads, 128]; v, out: [rows, heads, 128]; f:
    [rows, heads, 128] or [rows, heads]; b: [rows, heads]; a_log: float32
    [heads]; dt_bias: float32, f's shape without rows; state: float32
    [slots, heads, 128, 128] as [key, value].  scale multiplies q (128^-0.5
    unless given).  Column views of a packed projection output will do.
    """
    io, out, rows, H, Hk, pool = _operands(q, k, v, f, b, a_log, dt_bias, state, out, scale,
                                           l2norm)
    if slots.dtype is not torch.int32:
        raise TypeError("slots must be int32")
    if tokens < 1 or slots.dim() != 1 or slots.shape[0] * tokens != rows or \
            not slots.is_contiguous():
        raise ValueError("slots must be contiguous, one a request, with tokens rows each")
    _on_current_device(q, k, v, f, b, a_log, dt_bias, state, slots, out)
    rc = _lib().proj_delta_step(io, H, Hk, slots.shape[0], tokens,
                                slots.data_ptr(), pool, _stream_handle(stream))
    if rc:
        _check(rc, f"proj_delta_step(requests={slots.shape[0]}, tokens={tokens}, heads={H})")
    return out


class DeltaPlan:
    """A batch of sequences, made once and run for every layer: sequence i has
    lens[i] rows, packed one after another, and continues state[slots[i]]."""

    def __init__(self, lens, slots, *, heads: int, qk_heads: int | None = None, n_slots: int,
                 host_only: bool = False):
        lens, slots = [int(t) for t in lens], [int(t) for t in slots]
        if len(lens) != len(slots):
            raise ValueError("one slot a sequence")
        self.heads, self.n_slots = int(heads), int(n_slots)
        self.qk_heads = self.heads if qk_heads is None else int(qk_heads)
        n = len(lens)
        h = ctypes.c_void_p()
        rc = _lib().proj_delta_plan(self.heads, self.qk_heads, n,
                                    (ctypes.c_int * max(1, n))(*lens),
                                    (ctypes.c_int * max(1, n))(*slots), self.n_slots,
                                    PLAN_HOST_ONLY if host_only else 0, ctypes.byref(h))
        _check(rc, f"proj_delta_plan(heads={heads}, n={n})")
        self._h = h
        self.rows = int(_lib().proj_delta_plan_rows(h))
        self.device = None
        if not host_only:
            self.device = torch.cuda.current_device()

    def close(self):
        h, self._h = getattr(self, "_h", None), None
        if h:
            _lib().proj_delta_free(h)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def run(self, q, k, v, f, b, a_log, dt_bias, state, *, scale=None, l2norm: bool = True,
            out=None, stream=None):
        """The operands of delta_step, with the plan's rows (more rows may
        follow; theirs in out are left as they were, and out must then be
        given).  Updates state in place and returns out.  Without l2norm
        (keys of any length) the rows of a sequence run one by one, which is
        slow for long ones."""
        if out is None and q.dim() == 3 and q.shape[0] != self.rows:
            raise ValueError(f"{q.shape[0]} rows, the plan has {self.rows}: give out")
        io, out, rows, H, Hk, pool = _operands(q, k, v, f, b, a_log, dt_bias, state, out, scale,
                                               l2norm)
        if rows < self.rows:
            raise ValueError(f"{rows} rows, the plan has {self.rows}")
        if (H, Hk, pool) != (self.heads, self.qk_heads, self.n_slots):
            raise ValueError(f"{H} heads, {Hk} key heads and {pool} slots do not match the plan "
                             f"({self.heads}, {self.qk_heads}, {self.n_slots})")
        _same_device(q, k, v, f, b, a_log, dt_bias, state, out)
        if self.device is not None and q.device.index != self.device:
            raise ValueError(f"operands on cuda:{q.device.index}, the plan on cuda:{self.device}")
        rc = _lib().proj_delta_run(self._h, io, _stream_handle(stream))
        if rc:
            _check(rc, f"proj_delta_run(rows={self.rows}, heads={H})")
        return out
