"""Workloads of the layer operators: the norm with its 8-bit output, row codes, the 8-bit projection
and the gated delta rule in its recurrent and chunked forms.

Each case is one call (or the calls one call stands for) at sizes of a KDA decode layer: hidden size
7168, 96 heads of 128, the packed input projections 14560 x 7168 and 49376 x 7168, o_proj
7168 x 12288, and their 8-way shards.  The plain forms are elementary torch operations in 32 bits
(the inverse of a chunk's triangular matrix in 64).
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
HEAD = 128          # head size of keys and values
EPS = 1e-6
CHUNK = 32          # tokens a step of the plain chunked form


def listed():
    return [
        # the norm before a projection in a decode step of one request
        {"name": "norm decode 1", "op": "norm", "rows": 1, "dim": 7168, "residual": "bf16",
         "codes": False},
        # a long prompt's rows on a 32-bit residual stream, handed on in 8 bits
        {"name": "norm prompt 8 bits", "op": "norm", "rows": 8192, "dim": 7168,
         "residual": "fp32", "codes": True},
        # the o_proj input of a decode batch in 8 bits
        {"name": "codes decode 64", "op": "codes", "rows": 64, "dim": 12288},
        # a weight at load time: the packed DSA input projection, a scale a row
        {"name": "codes weight", "op": "codes", "rows": 14560, "dim": 7168},
        # an 8-way shard of the DSA input projection, one request: latency
        {"name": "proj shard 1", "op": "proj", "n": 1820, "k": 7168, "rows": 1},
        # the DSA input projection of a small decode batch
        {"name": "proj dsa 16", "op": "proj", "n": 14560, "k": 7168, "rows": 16},
        # the packed KDA input projection of a decode batch
        {"name": "proj kda 64", "op": "proj", "n": 49376, "k": 7168, "rows": 64},
        # o_proj of a large, ragged decode batch
        {"name": "proj o 251", "op": "proj", "n": 7168, "k": 12288, "rows": 251},
        # one request's decode step, all heads
        {"name": "step 1", "op": "step", "requests": 1, "live": 1, "tokens": 1, "heads": 96,
         "qk_heads": 96, "head_gate": False},
        # a verify step of four tokens a request, the batch padded to its captured size
        {"name": "step 64x4 padded", "op": "step", "requests": 64, "live": 61, "tokens": 4,
         "heads": 96, "qk_heads": 96, "head_gate": False},
        # a few short prompts on an 8-way shard of the heads, a gate a head, shared keys
        {"name": "prompts ragged", "op": "prompt", "lens": "1,700,1337", "heads": 12,
         "qk_heads": 6, "head_gate": True},
        # one long prompt, all heads
        {"name": "prompt 8192", "op": "prompt", "lens": "8192", "heads": 96, "qk_heads": 96,
         "head_gate": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "codes", "proj", "proj", "step", "step", "prompt", "prompt"])
    if op in ("norm", "codes"):
        dim = 8 * _log(rng, 8, 2048)
        rows = _log(rng, 1, max(1, min(16384, 8192 * 7168 // dim)))
        if op == "codes":
            return {"op": op, "rows": rows, "dim": dim}
        return {"op": op, "rows": rows, "dim": dim,
                "residual": rng.choice(["none", "bf16", "fp32"]), "codes": rng.random() < 0.5}
    if op == "proj":
        return {"op": op, "n": _log(rng, 33, 49376), "k": 16 * _log(rng, 4, 768),
                "rows": _log(rng, 1, 256)}
    qk = _log(rng, 1, 96)
    heads = qk * rng.choice([r for r in (1, 1, 2, 4) if r * qk <= 96])
    gate = rng.random() < 0.4
    if op == "step":
        tokens = rng.choice([1, 1, 1, 2, 3, 4, 7])
        requests = _log(rng, 1, 256)
        while requests * heads > 64 * 96:
            requests -= 1
        if requests * heads * tokens > 64 * 96 * 4:
            tokens = 1
        live = requests - (rng.randrange(min(4, requests)) if rng.random() < 0.5 else 0)
        return {"op": op, "requests": requests, "live": live, "tokens": tokens, "heads": heads,
                "qk_heads": qk, "head_gate": gate}
    n = rng.choice([1, 1, 2, 3, 5])
    total = _log(rng, 8, max(8, 8192 * 24 // heads // n))
    lens = [max(1, round(total * rng.uniform(0.25, 1.0))) for _ in range(n)]
    lens = [min(m, 8192) for m in lens]
    return {"op": op, "lens": ",".join(map(str, lens)), "heads": heads, "qk_heads": qk,
            "head_gate": gate}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, std=1.0, dtype=torch.bfloat16):
    """Normal values, drawn a block of rows at a time (large weights stay small in 32 bits)."""
    out = torch.empty(shape, dtype=dtype, device=DEV)
    rows = max(1, (1 << 26) // max(1, out[0].numel()))
    for r in range(0, shape[0], rows):
        part = out[r:r + rows]
        part.copy_(torch.randn(part.shape, generator=g, device=DEV) * std)
    return out


def _codes_of(x):
    """Symmetric 8-bit codes and scales of the rows of x, in 64 bits (inputs of the product)."""
    codes = torch.empty(x.shape, dtype=torch.int8, device=DEV)
    scale = torch.empty(x.shape[0], dtype=torch.float32, device=DEV)
    for r in range(0, x.shape[0], 4096):
        p = x[r:r + 4096].double()
        m = p.abs().amax(1)
        codes[r:r + 4096] = torch.round(p * (127.0 / m)[:, None]).to(torch.int8)
        scale[r:r + 4096] = (m / 127.0).float()
    return codes, scale


def _lens(case):
    return [int(t) for t in case["lens"].split(",")]


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case)
    if op in ("norm", "codes"):
        R, D = case["rows"], case["dim"]
        x = _randn(g, R, D)
        x[:, ::max(1, D // 5)] *= 12.0           # a few outlier channels, as activations have
        s["x"] = x
        if op == "norm":
            s["w"] = (1.0 + 0.1 * torch.randn(D, generator=g, device=DEV)).to(torch.bfloat16)
            if case["residual"] != "none":
                dt = torch.bfloat16 if case["residual"] == "bf16" else torch.float32
                s["residual_in"] = _randn(g, R, D, std=2.0, dtype=dt)
        return s
    if op == "proj":
        xc, xs = _codes_of(_randn(g, case["rows"], case["k"]))
        wc, ws = _codes_of(_randn(g, case["n"], case["k"], std=0.02))
        s.update(xc=xc, xs=xs, wc=wc, ws=ws)
        if own:
            import tp1_skinny_bf16_amd as tp
            s["plan"] = tp.PlanI8(case["n"], case["k"], [case["rows"]])
        return s
    H, Hk = case["heads"], case["qk_heads"]
    R = case["requests"] * case["tokens"] if op == "step" else sum(_lens(case))
    # the projection's output: q | k | v | b side by side in one row
    width = (2 * Hk + H) * HEAD + (H + 7) // 8 * 8
    row = _randn(g, R, width)
    o = Hk * HEAD
    s["q"] = row[:, :o].unflatten(1, (Hk, HEAD))
    s["k"] = row[:, o:2 * o].unflatten(1, (Hk, HEAD))
    s["v"] = row[:, 2 * o:2 * o + H * HEAD].unflatten(1, (H, HEAD))
    s["b"] = row[:, 2 * o + H * HEAD:2 * o + H * HEAD + H]
    gates = (H,) if case["head_gate"] else (H, HEAD)
    s["f"] = _randn(g, R, *gates)
    s["a_log"] = torch.log(1.0 + 15.0 * torch.rand(H, generator=g, device=DEV))
    dt = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand(gates, generator=g, device=DEV))
    s["dt_bias"] = dt + torch.log(-torch.expm1(-dt))   # the inverse of softplus
    n = case["requests"] if op == "step" else len(_lens(case))
    pool = n + 3
    s["state"] = _randn(g, pool, H, HEAD, HEAD, std=0.1, dtype=torch.float32)
    where = torch.randperm(pool, generator=torch.Generator().manual_seed(seed))[:n]
    if op == "step":
        where[case["live"]:] = -1                      # padding of the captured batch
        s["slots"] = where.to(torch.int32).to(DEV)
        s["out"] = torch.zeros((R, H, HEAD), dtype=torch.bfloat16, device=DEV)
        return s
    s["slots"] = where.to(DEV)
    L = -(-max(_lens(case)) // CHUNK) * CHUNK
    at = torch.full((n, L), R, dtype=torch.long)        # R: a row of zeros
    r0 = 0
    for i, m in enumerate(_lens(case)):
        at[i, :m] = torch.arange(r0, r0 + m)
        r0 += m
    s["at"] = at.to(DEV)
    if own:
        import tp1_skinny_bf16_amd as tp
        s["plan"] = tp.DeltaPlan(_lens(case), where.tolist(), heads=H, qk_heads=Hk, n_slots=pool)
    return s


# ------------------------------------------------------------------ plain forms

def _values(codes, scale):
    """What codes and scales stand for, in the type of the rows they were made from."""
    out = torch.empty(codes.shape, dtype=torch.bfloat16, device=codes.device)
    return torch.mul(codes, scale[:, None], out=out)


def _plain_codes(p):
    m = p.abs().amax(1, keepdim=True)
    codes = torch.round(p * (127.0 / m)).to(torch.int8)
    return codes, m[:, 0] / 127.0


def _plain_norm(s):
    h = s["x"].float()
    if s["residual"] != "none":
        h = h + s["residual_in"].float()
    rstd = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
    p = h * s["w"].float()
    got = {}
    if s["residual"] != "none":
        s["residual_in"].copy_(h)
        got["residual"] = s["residual_in"]
    if s["codes"]:
        codes, scale = _plain_codes(p)
        scale = scale * rstd[:, 0]
        got["values"] = _values(codes, scale)
        got["scale"] = scale
    else:
        got["y"] = (p * rstd).to(torch.bfloat16)
    return got


def _rule_inputs(s, dtype):
    """q, k, v, log decay and beta a row and value head, in `dtype`."""
    rep = s["heads"] // s["qk_heads"]

    def unit(t):
        t = t.to(dtype)
        return t * torch.rsqrt(t.square().sum(-1, keepdim=True) + EPS)

    q = (unit(s["q"]) * HEAD ** -0.5).repeat_interleave(rep, 1)
    k = unit(s["k"]).repeat_interleave(rep, 1)
    v = s["v"].to(dtype)
    z = s["f"].to(dtype) + s["dt_bias"].to(dtype)
    soft = torch.clamp(z, min=0) + torch.log1p(torch.exp(-z.abs()))
    rate = torch.exp(s["a_log"].to(dtype))
    g = -rate * soft if s["head_gate"] else -rate[:, None] * soft
    if s["head_gate"]:
        g = g[..., None].expand(v.shape)
    beta = 1.0 / (1.0 + torch.exp(-s["b"].to(dtype)))
    return q, k, v, g, beta


def _token(S, q, k, v, g, beta):
    """One token of the rule on states [.., key, value]; returns the new states and the output."""
    S = S * torch.exp(g)[..., None]
    u = beta[..., None] * (v - (S * k[..., None]).sum(-2))
    S = S + k[..., None] * u[..., None, :]
    return S, (S * q[..., None]).sum(-2)


def _plain_step(s, dtype=torch.float32):
    live, T = s["live"], s["tokens"]
    q, k, v, g, beta = _rule_inputs(s, dtype)
    slots = s["slots"][:live].long()
    S = s["state"][slots].to(dtype)
    out = torch.zeros(s["out"].shape, dtype=dtype, device=DEV)
    for t in range(T):
        at = slice(t, live * T, T)
        S, out[at] = _token(S, q[at], k[at], v[at], g[at], beta[at])
    return slots, S, out


def _padded(s, t):
    """Rows of t laid out [sequence, token, ..], zeros past each sequence's end."""
    t = torch.cat([t, torch.zeros_like(t[:1])])
    return t[s["at"]]


def _plain_prompt(s):
    q, k, v, g, beta = (_padded(s, t) for t in _rule_inputs(s, torch.float32))
    n, L, H = beta.shape
    S = s["state"][s["slots"]]
    eye = torch.eye(CHUNK, dtype=torch.float64, device=DEV)
    keep = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=DEV).tril()
    out = torch.empty(n, L, H, HEAD, device=DEV)
    for c in range(0, L, CHUNK):
        qc, kc, vc, gc = (t[:, c:c + CHUNK].transpose(1, 2) for t in (q, k, v, g))
        bc = beta[:, c:c + CHUNK].transpose(1, 2)[..., None]
        G = gc.cumsum(2)
        D = torch.exp(torch.clamp(G[:, :, :, None] - G[:, :, None], max=0)) * kc[:, :, None]
        A = (D * kc[:, :, :, None]).sum(-1) * keep
        P = (D * qc[:, :, :, None]).sum(-1) * keep
        # (1 + N)^-1 of the strictly lower triangular N, by squaring: N^32 = 0
        N = -(bc * A).double().tril(-1)
        inv = eye + N
        for _ in range(4):
            N = N @ N
            inv = inv + N @ inv
        u = inv.float() @ (bc * (vc - (kc * torch.exp(G)) @ S))
        o = (qc * torch.exp(G)) @ S + P @ u
        out[:, c:c + CHUNK] = o.transpose(1, 2)
        last = G[:, :, -1:]
        S = S * torch.exp(last).transpose(2, 3) + \
            (kc * torch.exp(last - G)).transpose(2, 3).contiguous() @ u
    return S, out[s["at"] < s["q"].shape[0]]


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["op"]
    if own:
        import tp1_skinny_bf16_amd as tp
        if op == "norm":
            res = s.get("residual_in")
            got = {} if res is None else {"residual": res}
            if s["codes"]:
                codes, scale = tp.rms_norm_i8(s["x"], s["w"], residual=res, eps=EPS)
                return {**got, "values": _values(codes, scale), "scale": scale}
            return {**got, "y": tp.rms_norm(s["x"], s["w"], residual=res, eps=EPS)}
        if op == "codes":
            codes, scale = tp.quant_rows(s["x"])
            return {"values": _values(codes, scale), "scale": scale}
        if op == "proj":
            return {"y": s["plan"].run(s["xc"], s["xs"], s["wc"], s["ws"])}
        if op == "step":
            tp.delta_step(s["q"], s["k"], s["v"], s["f"], s["b"], s["a_log"], s["dt_bias"],
                          s["state"], s["slots"], tokens=s["tokens"], out=s["out"])
            return {"out": s["out"], "state": s["state"]}
        out = s["plan"].run(s["q"], s["k"], s["v"], s["f"], s["b"], s["a_log"], s["dt_bias"],
                            s["state"])
        return {"out": out, "state": s["state"]}
    if op == "norm":
        return _plain_norm(s)
    if op == "codes":
        codes, scale = _plain_codes(s["x"].float())
        return {"values": _values(codes, scale), "scale": scale}
    if op == "proj":
        acc = s["xc"].float() @ s["wc"].float().t()
        return {"y": (acc * s["xs"][:, None] * s["ws"]).to(torch.bfloat16)}
    if op == "step":
        slots, S, out = _plain_step(s)
        s["state"][slots] = S
        return {"out": out.to(torch.bfloat16), "state": s["state"]}
    S, out = _plain_prompt(s)
    s["state"][s["slots"]] = S
    return {"out": out.to(torch.bfloat16), "state": s["state"]}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "codes"):
        h = s["x"].double()
        got, norm = {}, 1.0
        if op == "norm":
            if case["residual"] != "none":
                h += s["residual_in"]
                got["residual"] = h.clone()
            norm = 1.0 / torch.sqrt((h * h).sum(1) / h.shape[1] + EPS)
            h *= s["w"].double()
            if not case["codes"]:
                got["y"] = h * norm[:, None]
                return got
        top = h.abs().max(1).values
        scale = top * norm / 127.0
        got["values"] = torch.round(h / (top / 127.0)[:, None]) * scale[:, None]
        got["scale"] = scale
        return got
    if op == "proj":
        y = torch.matmul(s["wc"].double(), s["xc"].double().t())
        return {"y": (y * s["ws"].double()[:, None] * s["xs"].double()).t()}
    # the rule token by token, sequences side by side
    rep = case["heads"] // case["qk_heads"]
    H = case["heads"]
    q, k, v = (s[t].double() for t in "qkv")
    q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + EPS) / math.sqrt(HEAD)
    k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + EPS)
    of = torch.arange(H, device=DEV) // rep
    z = s["f"].double() + s["dt_bias"].double()
    rate = s["a_log"].double().exp()
    decay = torch.exp(-rate.reshape(H, *([1] * (z.dim() - 2))) * torch.logaddexp(z, torch.zeros_like(z)))
    decay = decay.reshape(decay.shape[0], H, -1)
    beta = torch.sigmoid(s["b"].double())
    state = s["state"].double()
    out = torch.zeros(q.shape[0], H, HEAD, dtype=torch.float64, device=DEV)
    if op == "step":
        rows = torch.arange(case["live"], device=DEV)[:, None] * case["tokens"] + \
            torch.arange(case["tokens"], device=DEV)
        ends = [case["tokens"]] * case["live"]
        slots = s["slots"][:case["live"]].long()
    else:
        rows, ends, slots = s["at"], _lens(case), s["slots"]
    ends_dev = torch.tensor(ends, device=DEV)
    for t in range(max(ends)):
        on = torch.nonzero(ends_dev > t)[:, 0] if len(set(ends)) > 1 else slice(None)
        r, sl = rows[on, t], slots[on]
        S = state[sl] * decay[r][..., None]
        kt, qt = k[r][:, of], q[r][:, of]
        u = beta[r][..., None] * (v[r] - torch.einsum("nhkv,nhk->nhv", S, kt))
        S = S + torch.einsum("nhk,nhv->nhkv", kt, u)
        state[sl] = S
        out[r] = torch.einsum("nhkv,nhk->nhv", S, qt)
    return {"out": out, "state": state}


def work(case):
    op = case["op"]
    if op in ("norm", "codes"):
        n = case["rows"] * case["dim"]
        per = 2 + (1 if op == "codes" or case["codes"] else 2)
        if op == "norm":
            per += {"none": 0, "bf16": 4, "fp32": 8}[case["residual"]]
        extra = 4 * case["rows"] + (2 * case["dim"] if op == "norm" else 0)
        return {"bytes": n * per + extra, "flops": 6 * n}
    if op == "proj":
        n, k, b = case["n"], case["k"], case["rows"]
        return {"bytes": n * k + b * k + 4 * (n + b) + 2 * b * n, "flops": 2 * n * k * b}
    H, Hk = case["heads"], case["qk_heads"]
    if op == "step":
        seqs, rows = case["live"], case["live"] * case["tokens"]
    else:
        seqs, rows = len(_lens(case)), sum(_lens(case))
    gate = H if case["head_gate"] else H * HEAD
    row = 2 * (2 * Hk * HEAD + 2 * H * HEAD + gate + H)
    return {"bytes": rows * row + seqs * H * HEAD * HEAD * 8 + 4 * (H + gate),
            "flops": rows * H * 7 * HEAD * HEAD}
