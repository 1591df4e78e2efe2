"""Plain 64-bit forms of the layer operators (CPU), and the inputs of their tests."""
from __future__ import annotations

import math

import torch

HEAD = 128
U32 = 2.0 ** -24      # half a step of float32, relative
U16 = 2.0 ** -8       # of bfloat16


def norm(x, w, residual, eps):
    """(h, y) of proj_rms_norm in 64 bits."""
    h = x.double() if residual is None else x.double() + residual.double()
    y = h * w.double() / torch.sqrt(h.square().mean(1, keepdim=True) + eps)
    return h, y


def delta(q, k, v, f, b, a_log, dt_bias, state, seqs, *, scale=HEAD ** -0.5, l2norm=True):
    """The rule token by token in 64 bits.  seqs: (first row, rows, slot) each,
    run in order; returns (out [rows, H, 128], state), zeros in rows of no
    sequence."""
    q, k, v, f, b = (t.double() for t in (q, k, v, f, b))
    a_log, dt_bias, state = a_log.double(), dt_bias.double(), state.double().clone()
    H, rep = v.shape[1], v.shape[1] // q.shape[1]
    if l2norm:
        q = q / torch.sqrt(q.square().sum(-1, keepdim=True) + 1e-6)
        k = k / torch.sqrt(k.square().sum(-1, keepdim=True) + 1e-6)
    q = (q * scale).repeat_interleave(rep, 1)
    k = k.repeat_interleave(rep, 1)
    z = f + dt_bias
    soft = torch.logaddexp(z, torch.zeros_like(z))
    rate = a_log.exp() if f.dim() == 2 else a_log.exp()[:, None]
    a = torch.exp(-rate * soft)
    a = a[..., None].expand(v.shape) if f.dim() == 2 else a
    beta = torch.sigmoid(b)
    out = torch.zeros(v.shape, dtype=torch.float64)
    for r0, n, slot in seqs:
        S = state[slot]
        for r in range(r0, r0 + n):
            S = S * a[r][:, :, None]
            u = beta[r][:, None] * (v[r] - torch.einsum("hkv,hk->hv", S, k[r]))
            S = S + torch.einsum("hk,hv->hkv", k[r], u)
            out[r] = torch.einsum("hkv,hk->hv", S, q[r])
        state[slot] = S
    return out, state


def delta_inputs(rows, heads, qk_heads, head_gate, slots, seed, gate_std=1.0):
    """CPU tensors: columns of one packed row (q | k | v | b), f, a_log, dt_bias, state."""
    g = torch.Generator().manual_seed(seed)
    width = (2 * qk_heads + heads) * HEAD + (heads + 7) // 8 * 8
    row = torch.randn(rows, width, generator=g).to(torch.bfloat16)
    gates = (heads,) if head_gate else (heads, HEAD)
    f = (gate_std * torch.randn(rows, *gates, generator=g)).to(torch.bfloat16)
    a_log = torch.log(1.0 + 15.0 * torch.rand(heads, generator=g))
    dt = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand(gates, generator=g))
    dt_bias = dt + torch.log(-torch.expm1(-dt))
    state = 0.1 * torch.randn(slots, heads, HEAD, HEAD, generator=g)
    return {"row": row, "f": f, "a_log": a_log, "dt_bias": dt_bias, "state": state,
            "heads": heads, "qk_heads": qk_heads}


def columns(c):
    """(q, k, v, b): views of the packed rows of delta_inputs."""
    o, H = c["qk_heads"] * HEAD, c["heads"]
    row = c["row"]
    return (row[:, :o].unflatten(1, (c["qk_heads"], HEAD)),
            row[:, o:2 * o].unflatten(1, (c["qk_heads"], HEAD)),
            row[:, 2 * o:2 * o + H * HEAD].unflatten(1, (H, HEAD)),
            row[:, 2 * o + H * HEAD:2 * o + H * HEAD + H])
