"""A stack of KDA layers in 8 bits over the layer operators.

On the vLLM API page "vllm.models.kimi_k3.nvidia.specialized_decode.runtime.
dep" (section "DepKda") a KDA layer projects its rows, runs the recurrence
over its states and projects back; the loop around it ("…runtime.hybrid",
section "HybridStep.run") normalises the residual stream before each layer.
Here a layer is, for x [B, D] and the residual stream r [B, D]:

    r += x; codes of rms_norm(r) * w                     rms_norm_i8
    q | k | v | f | b = codes . w_in^T                   PlanI8
    f = f . w_f^T  (low rank -> a gate a channel)        Plan (BF16)
    o = the gated delta rule over the states             delta_step or a DeltaPlan
    codes of o;  x = codes . w_o^T                       quant_rows, PlanI8

LayerStack runs the two projections of a layer in BF16 with nothing between
them.  The layer's short convolution and output gate are not part of it.
"""
from __future__ import annotations

import dataclasses

import torch

from ._binding import PROJ_EBATCH, Plan, ProjError
from .delta import HEAD, delta_step
from .norm import quant_rows, rms_norm_i8
from .proj_i8 import PlanI8


@dataclasses.dataclass
class KdaLayer:
    """One layer's weights: norm [D] BF16; w_in int8 [N_in, D] and w_in_scale
    [N_in], rows q | k | v | f | b (then padding to a multiple of 8); w_f BF16
    [heads * 128, rank]; a_log [heads], dt_bias [heads, 128] FP32; w_o int8
    [D, heads * 128] and w_o_scale [D]."""
    norm: torch.Tensor
    w_in: torch.Tensor
    w_in_scale: torch.Tensor
    w_f: torch.Tensor
    a_log: torch.Tensor
    dt_bias: torch.Tensor
    w_o: torch.Tensor
    w_o_scale: torch.Tensor


class KdaStack:
    """Layers of one shape for batches of up to max(batches) rows."""

    def __init__(self, layers, batches, *, heads: int, qk_heads: int | None = None,
                 eps: float = 1e-6):
        self.layers = list(layers)
        if not self.layers:
            raise ValueError("a stack needs at least one layer")
        first = self.layers[0]
        self.heads, self.eps = int(heads), eps
        self.qk_heads = self.heads if qk_heads is None else int(qk_heads)
        self.N_in, self.D = (int(n) for n in first.w_in.shape)
        self.rank = int(first.w_f.shape[1])
        used = (2 * self.qk_heads + self.heads) * HEAD + self.rank + self.heads
        if self.N_in < used or self.N_in % 8 or self.rank % 8:
            raise ValueError(f"w_in must have at least {used} rows, a multiple of 8, and the "
                             "rank of w_f must be one")
        for i, ly in enumerate(self.layers):
            if ly.w_in.shape != (self.N_in, self.D) or \
                    ly.w_f.shape != (self.heads * HEAD, self.rank) or \
                    ly.w_o.shape != (self.D, self.heads * HEAD):
                raise ValueError(f"layer {i} does not have the shape of layer 0")
        self.most = max(batches)
        self.in_plan = PlanI8(self.N_in, self.D, batches)
        self.f_plan = Plan(self.heads * HEAD, self.rank, batches)
        self.o_plan = PlanI8(self.D, self.heads * HEAD, batches)

    def buffers(self, B: int):
        """What a layer writes, for run(..., buf=): one set serves every layer."""
        dev, w = self.layers[0].w_in.device, self.heads * HEAD

        def new(shape, dtype=torch.bfloat16):
            return torch.empty(shape, dtype=dtype, device=dev)
        return {"codes": new((B, self.D), torch.int8), "scale": new((B,), torch.float32),
                "y": new((B, self.N_in)), "f": new((B, w)), "o": new((B, self.heads, HEAD)),
                "o_codes": new((B, w), torch.int8), "o_scale": new((B,), torch.float32),
                "x": new((B, self.D))}

    def run_layer(self, i: int, x, residual, state, buf, *, slots=None, tokens: int = 1,
                  plan=None, stream=None):
        """Layer i on x [B, D]: updates residual and state, returns buf["x"]."""
        ly, B = self.layers[i], x.shape[0]
        rms_norm_i8(x, ly.norm, residual=residual, eps=self.eps, codes=buf["codes"],
                    scale=buf["scale"], stream=stream)
        y = self.in_plan.run(buf["codes"], buf["scale"], ly.w_in, ly.w_in_scale, buf["y"],
                             stream=stream)
        hq, h = self.qk_heads * HEAD, self.heads * HEAD
        q = y[:, :hq].unflatten(1, (self.qk_heads, HEAD))
        k = y[:, hq:2 * hq].unflatten(1, (self.qk_heads, HEAD))
        v = y[:, 2 * hq:2 * hq + h].unflatten(1, (self.heads, HEAD))
        c = 2 * hq + h
        f = self.f_plan.run(y[:, c:c + self.rank], ly.w_f, buf["f"], stream=stream)
        b = y[:, c + self.rank:c + self.rank + self.heads]
        args = (q, k, v, f.view(B, self.heads, HEAD), b, ly.a_log, ly.dt_bias, state)
        if plan is None:
            delta_step(*args, slots, tokens=tokens, out=buf["o"], stream=stream)
        else:
            plan.run(*args, out=buf["o"], stream=stream)
        quant_rows(buf["o"].view(B, h), codes=buf["o_codes"], scale=buf["o_scale"],
                   stream=stream)
        return self.o_plan.run(buf["o_codes"], buf["o_scale"], ly.w_o, ly.w_o_scale, buf["x"],
                               stream=stream)

    def run(self, x, residual, states, *, slots=None, tokens: int = 1, plan=None, buf=None,
            stream=None):
        """Every layer on x [B, D]; returns the last layer's output (to be
        added to the residual by whatever follows).  states: one state pool a
        layer.  slots (int32 on the device) and tokens as delta_step takes
        them, or a DeltaPlan for sequences of up to the batch's rows."""
        if (slots is None) == (plan is None):
            raise ValueError("give slots (a decode step) or plan (sequences)")
        if len(states) != len(self.layers):
            raise ValueError("one state pool a layer")
        # before the first layer changes the residual
        if x.shape[0] > self.most:
            raise ProjError(PROJ_EBATCH, f"{x.shape[0]} rows, planned for {self.most}")
        if plan is not None and plan.rows != x.shape[0]:
            raise ValueError(f"{x.shape[0]} rows, the plan has {plan.rows}")
        if slots is not None and slots.shape[0] * tokens != x.shape[0]:
            raise ValueError(f"{x.shape[0]} rows, the slots have {slots.shape[0]} x {tokens}")
        buf = self.buffers(x.shape[0]) if buf is None else buf
        for i, state in enumerate(states):
            x = self.run_layer(i, x, residual, state, buf, slots=slots, tokens=tokens, plan=plan,
                               stream=stream)
        return x

    def close(self):
        for p in (self.in_plan, self.f_plan, self.o_plan):
            p.close()
