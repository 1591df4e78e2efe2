"""The decode projection in 8-bit integers (argument marshalling; the work is
proj_i8_run): Plan's counterpart for weights held as codes with a scale per
output channel, half the bytes a BF16 weight streams."""
from __future__ import annotations

import ctypes

import torch

from ._binding import PLAN_HOST_ONLY, Tactic, _check, _lib, _stream_handle, _Tactic


class PlanI8:
    """A plan for an N x K int8 weight and a list of batch sizes."""

    def __init__(self, N: int, K: int, batches, *, host_only: bool = False):
        self.N, self.K = int(N), int(K)
        self.batches = tuple(int(b) for b in batches)
        arr = (ctypes.c_int * max(1, len(self.batches)))(*self.batches)
        h = ctypes.c_void_p()
        rc = _lib().proj_i8_plan(self.N, self.K, arr, len(self.batches),
                                 PLAN_HOST_ONLY if host_only else 0, ctypes.byref(h))
        _check(rc, f"proj_i8_plan(N={N}, K={K}, batches={self.batches})")
        self._h = h
        self.host_only = host_only
        self.device = None
        if not host_only:
            self.device = torch.cuda.current_device()

    def close(self):
        h, self._h = getattr(self, "_h", None), None
        if h:
            _lib().proj_i8_free(h)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    @property
    def workspace_bytes(self) -> int:
        return int(_lib().proj_i8_plan_workspace_bytes(self._h))

    def tactic(self, B: int):
        """(Tactic, bin) proj_i8_run would use for batch B."""
        t, b = _Tactic(), ctypes.c_int()
        _check(_lib().proj_i8_plan_tactic(self._h, int(B), ctypes.byref(t), ctypes.byref(b)),
               f"proj_i8_plan_tactic(B={B})")
        return Tactic(*[getattr(t, n) for n, _ in _Tactic._fields_]), b.value

    def set_tactic(self, bin_: int, tactic: Tactic):
        c = tactic._c()
        _check(_lib().proj_i8_plan_set_tactic(self._h, int(bin_), ctypes.byref(c)),
               f"proj_i8_plan_set_tactic(bin={bin_}, {tactic})")

    def run_ptr(self, B: int, x: int, ldx: int, x_scale: int, w: int, w_scale: int, y: int,
                stream: int = 0) -> int:
        """Raw call: returns the status code instead of raising."""
        return _lib().proj_i8_run(self._h, B, x, ldx, x_scale, w, w_scale, y, stream)

    def run(self, x, x_scale, W, w_scale, out=None, *, stream=None):
        """out[B, N] = (x . W^T) * x_scale[:, None] * w_scale, BF16, of int8
        codes x [B, K] (rows may have a stride > K) and W [N, K]."""
        if x.dtype is not torch.int8 or W.dtype is not torch.int8:
            raise TypeError("x and W must be int8")
        if x_scale.dtype is not torch.float32 or w_scale.dtype is not torch.float32:
            raise TypeError("the scales must be float32")
        N, K = self.N, self.K
        if x.dim() != 2 or x.shape[1] != K or W.shape != (N, K):
            raise ValueError(f"shapes x{tuple(x.shape)} W{tuple(W.shape)} do not "
                             f"match the plan ({N} x {K})")
        B = x.shape[0]
        ldx, one = x.stride()
        if (one != 1 and B > 0) or not W.is_contiguous():
            raise ValueError("x needs unit column stride and W must be contiguous")
        if B > 1 and ldx < K:
            raise ValueError("the rows of x overlap")
        if x_scale.shape != (B,) or w_scale.shape != (N,) or \
                not (x_scale.is_contiguous() and w_scale.is_contiguous()):
            raise ValueError("the scales must be contiguous, one a row of x and of W")
        if out is None:
            out = x.new_empty((B, N), dtype=torch.bfloat16)
        elif out.shape != (B, N) or not out.is_contiguous() or out.dtype is not torch.bfloat16:
            raise ValueError("out must be a contiguous bfloat16 [B, N] tensor")
        dev = x.get_device()
        if dev < 0 or not (dev == W.get_device() == x_scale.get_device() ==
                           w_scale.get_device() == out.get_device()):
            raise ValueError("every operand must be a device tensor, all on one device")
        if self.device is not None and dev != self.device:
            raise ValueError(f"operands on cuda:{dev}, the plan on cuda:{self.device}")
        rc = self.run_ptr(B, x.data_ptr(), ldx if B > 1 else K, x_scale.data_ptr(),
                          W.data_ptr(), w_scale.data_ptr(), out.data_ptr(),
                          _stream_handle(stream))
        if rc:
            _check(rc, f"proj_i8_run(B={B})")
        return out
