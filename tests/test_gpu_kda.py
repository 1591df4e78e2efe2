"""GPU tests of KdaStack: the layer operators run together.  Every stage is
checked on the values the stack itself handed it (so errors do not pile up),
against 64 bits with the stage's own tolerance; the whole is compared with
the stages called one by one, and replayed as a graph."""
import pytest
import torch

import tp1_skinny_bf16_amd as tp
from gpu_util import DEV, say
from layer_ref import HEAD, U16, U32, delta, norm

pytestmark = pytest.mark.gpu

D, RANK = 512, 32


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    torch.cuda.set_device(DEV)


def make(layers, heads, qk, batches, seed=3):
    g = torch.Generator().manual_seed(seed)
    n_in = ((2 * qk + heads) * HEAD + RANK + heads + 7) // 8 * 8

    def codes(n, k):
        w = (torch.randn(n, k, generator=g) / k ** 0.5).to(torch.bfloat16).to(DEV)
        return tp.quant_rows(w)
    out = []
    for _ in range(layers):
        wi, si = codes(n_in, D)
        wo, so = codes(D, heads * HEAD)
        out.append(tp.KdaLayer(
            norm=(1 + 0.1 * torch.randn(D, generator=g)).to(torch.bfloat16).to(DEV),
            w_in=wi, w_in_scale=si,
            w_f=(torch.randn(heads * HEAD, RANK, generator=g) / RANK ** 0.5)
            .to(torch.bfloat16).to(DEV),
            a_log=torch.log(1 + 15 * torch.rand(heads, generator=g)).to(DEV),
            dt_bias=(-4 + torch.randn(heads, HEAD, generator=g)).to(DEV),
            w_o=wo, w_o_scale=so))
    return tp.KdaStack(out, batches, heads=heads, qk_heads=qk)


def product(codes, scale, w, ws):
    acc = (codes.cpu().double() @ w.cpu().double().t()).to(torch.float32)
    return (acc * (scale.cpu()[:, None] * ws.cpu())).to(torch.bfloat16)


@pytest.mark.parametrize("heads,qk,B,tokens,lens", [(4, 2, 6, 2, None), (3, 3, 5, 1, None),
                                                    (2, 2, 90, 0, [70, 20])])
def test_every_stage_of_a_layer(heads, qk, B, tokens, lens):
    stack = make(2, heads, qk, [8, 128])
    g = torch.Generator().manual_seed(9)
    x = torch.randn(B, D, generator=g).to(torch.bfloat16)
    r = torch.randn(B, D, generator=g)
    n = len(lens) if lens else B // tokens
    states = [0.1 * torch.randn(n + 1, heads, HEAD, HEAD, generator=g) for _ in range(2)]
    if lens:
        plan = tp.DeltaPlan(lens, [1, 0], heads=heads, qk_heads=qk, n_slots=n + 1)
        how = {"plan": plan}
        seqs = [(0, lens[0], 1), (lens[0], lens[1], 0)]
    else:
        slots = torch.arange(n, 0, -1, dtype=torch.int32)
        how = {"slots": slots.to(DEV), "tokens": tokens}
        seqs = [(i * tokens, tokens, int(s)) for i, s in enumerate(slots)]
    buf = stack.buffers(B)
    xd, rd = x.to(DEV), r.to(DEV)
    sd = [s.to(DEV) for s in states]
    for i, ly in enumerate(stack.layers):
        before = (xd.cpu(), rd.cpu(), sd[i].cpu())
        stack.run_layer(i, xd.clone(), rd, sd[i], buf, **how)
        torch.cuda.synchronize()
        h, y = norm(before[0], ly.norm.cpu(), before[1], stack.eps)
        assert ((rd.cpu().double() - h).abs() / h.abs().clamp(min=1e-30)).max() <= U32
        want = y.abs().amax(1) / 127
        assert ((buf["scale"].cpu().double() - want).abs() / want).max() <= 40 * U32
        t = y / want[:, None]
        assert (buf["codes"].cpu().double() - t).abs().max() <= 0.5 + 127 * 8 * U32
        got = buf["y"].cpu()
        assert torch.equal(got, product(buf["codes"], buf["scale"], ly.w_in, ly.w_in_scale))
        hq, hv = qk * HEAD, heads * HEAD
        c = 2 * hq + hv
        f = got[:, c:c + RANK].double() @ ly.w_f.cpu().double().t()
        err = (buf["f"].cpu().double() - f).abs() - U16 * f.abs()
        # FP32 sums of RANK products
        tol = RANK * 2 * U32 * (got[:, c:c + RANK].double().abs() @
                                ly.w_f.cpu().double().abs().t())
        assert bool((err <= tol).all())
        o, S = delta(got[:, :hq].unflatten(1, (qk, HEAD)), got[:, hq:2 * hq].unflatten(
            1, (qk, HEAD)), got[:, 2 * hq:c].unflatten(1, (heads, HEAD)),
            buf["f"].cpu().view(B, heads, HEAD), got[:, c + RANK:c + RANK + heads],
            ly.a_log.cpu(), ly.dt_bias.cpu(), before[2], seqs)
        rel = ((sd[i].cpu().double() - S).norm() / S.norm()).item()
        M = S.norm(dim=2).max().item() + got[:, 2 * hq:c].abs().max().item()
        od = (buf["o"].cpu().double() - o).abs() - U16 * o.abs()
        say(f"[kda layer {i} H={heads}/{qk} B={B}] state rel {rel:.1e}, out beyond rounding "
            f"{od.max().item():.1e}")
        assert rel <= 2.0 ** -20
        assert od.max().item() <= 256 * max(lens or [tokens]) * U32 * M
        oc, os_ = tp.quant_rows(buf["o"].view(B, hv))
        assert torch.equal(oc, buf["o_codes"]) and torch.equal(os_, buf["o_scale"])
        assert torch.equal(buf["x"].cpu(), product(oc, os_, ly.w_o, ly.w_o_scale))
        xd = buf["x"].clone()
    # the whole at once
    rd2, sd2 = r.to(DEV), [s.to(DEV) for s in states]
    out = stack.run(x.to(DEV), rd2, sd2, **how)
    torch.cuda.synchronize()
    assert torch.equal(out, xd) and torch.equal(rd2, rd)
    assert all(torch.equal(a, b) for a, b in zip(sd, sd2))
    stack.close()


def test_a_captured_step_replays():
    heads, B = 4, 5
    stack = make(3, heads, heads, [8])
    g = torch.Generator().manual_seed(2)
    x = torch.randn(B, D, generator=g).to(torch.bfloat16).to(DEV)
    r = torch.randn(B, D, generator=g).to(DEV)
    states = [0.1 * torch.randn(B, heads, HEAD, HEAD, generator=g).to(DEV) for _ in range(3)]
    slots = torch.tensor([2, 0, 3, 1, -1], dtype=torch.int32, device=DEV)
    buf = stack.buffers(B)
    xin, rin, sin = x.clone(), r.clone(), [s.clone() for s in states]
    stack.run(xin, rin, sin, slots=slots, buf=buf)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = stack.run(xin, rin, sin, slots=slots, buf=buf)
    rin.copy_(r)
    for a, b in zip(sin, states):
        a.copy_(b)
    eager = stack.buffers(B)
    for step in range(4):
        want = stack.run(x, r, states, slots=slots, buf=eager).clone()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(rin, r)
        assert all(torch.equal(a, b) for a, b in zip(sin, states))
        x.mul_(-0.5)
        xin.copy_(x)
        slots.copy_(torch.roll(slots, 1))
    stack.close()


def test_refusals():
    stack = make(1, 2, 2, [4])
    x = torch.zeros(3, D, dtype=torch.bfloat16, device=DEV)
    r = torch.zeros(3, D, device=DEV)
    st = [torch.zeros(4, 2, HEAD, HEAD, device=DEV)]
    slots = torch.zeros(3, dtype=torch.int32, device=DEV)
    plan = tp.DeltaPlan([2], [0], heads=2, n_slots=4)
    for kw in ({}, {"slots": slots, "plan": plan}, {"plan": plan}, {"slots": slots[:2]}):
        with pytest.raises(ValueError):
            stack.run(x, r, st, **kw)
    with pytest.raises(ValueError):
        stack.run(x, r, st * 2, slots=slots)
    big = torch.zeros(5, D, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(tp.ProjError):                      # above the planned batches
        stack.run(big, torch.zeros(5, D, device=DEV), st,
                  slots=torch.zeros(5, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        tp.KdaStack([], [4], heads=2)
    with pytest.raises(ValueError):
        tp.KdaStack(stack.layers, [4], heads=3)


def test_refusals_leave_the_residual_as_it_was():
    stack = make(1, 2, 2, [8])
    state = [torch.zeros(9, 2, HEAD, HEAD, device=DEV)]
    slots = torch.arange(8, dtype=torch.int32, device=DEV)
    for rows, how in ((9, {"slots": torch.arange(9, dtype=torch.int32, device=DEV)}),
                      (8, {"slots": slots[:7]}), (8, {"slots": slots, "tokens": 2}),
                      (8, {"plan": tp.DeltaPlan([7], [0], heads=2, n_slots=9)}), (8, {})):
        x = torch.ones(rows, D, dtype=torch.bfloat16, device=DEV)
        r = torch.ones(rows, D, device=DEV)
        with pytest.raises((ValueError, tp.ProjError)):
            stack.run(x, r, state, **how)
        torch.cuda.synchronize()
        assert bool((r == 1).all())
