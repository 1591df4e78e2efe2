"""GPU tests of the 8-bit projection.  The integer sum is exact and the rest
is three IEEE roundings in a fixed order, so every output is compared bit for
bit with the same three roundings of the exact sum on the CPU."""
import pytest
import torch

import tp1_skinny_bf16_amd as tp
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    torch.cuda.set_device(DEV)


def case(B, N, K, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(-128, 128, (B, K + pad), generator=g, dtype=torch.int8)[:, :K]
    w = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int8)
    xs = torch.rand(B, generator=g) * 0.1
    ws = torch.rand(N, generator=g) * 1e-3
    return x, xs, w, ws


def expected(x, xs, w, ws):
    # float64 holds the sums exactly: 128 * 128 * K < 2^53
    acc = (x.double() @ w.double().t()).to(torch.float32)
    return (acc * (xs[:, None] * ws[None, :])).to(torch.bfloat16)


def device_rows(x):
    if x.is_contiguous():
        return x.to(DEV)
    big = torch.full((x.shape[0], x.stride(0)), 99, dtype=torch.int8, device=DEV)
    big[:, :x.shape[1]] = x.to(DEV)
    return big[:, :x.shape[1]]


def run(plan, x, xs, w, ws):
    y = plan.run(device_rows(x), xs.to(DEV), w.to(DEV), ws.to(DEV))
    torch.cuda.synchronize()
    return y.cpu()


def same(label, got, want):
    bad = (got.view(torch.int16) != want.view(torch.int16)).sum().item()
    say(f"[{label}] {got.numel()} outputs, {bad} differ")
    assert bad == 0


@pytest.mark.parametrize("N,K,pad", [(33, 16, 0), (1, 64, 16), (1000, 1040, 32), (777, 2064, 0),
                                     (1820, 7168, 0), (20, 12288, 16), (5000, 208, 0)])
def test_every_bin(N, K, pad):
    plan = tp.PlanI8(N, K, [1, 2, 4, 8, 16, 32, 64, 128, 256])
    x, xs, w, ws = case(256, N, K, seed=N + K, pad=pad)
    for B in (1, 3, 16, 17, 32, 50, 64, 100, 128, 251, 256):
        same(f"i8 {N}x{K} B={B}", run(plan, x[:B], xs[:B], w, ws),
             expected(x[:B], xs[:B], w, ws))


def instances():
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = open(os.path.join(root, "tp1_skinny_bf16_amd", "csrc", "proj_i8.hip")).read()
    blk = src[src.index("TP1_I8_INSTANCES(X)"):]
    blk = blk[:blk.index("\n\n")]
    return [tuple(map(int, m)) for m in
            re.findall(r"X\((\d+), (\d+), (\d+), (\d+), (\d+), (\d+), (\d+)\)", blk)]


@pytest.mark.parametrize("inst", instances())
def test_every_instance_split_and_order(inst):
    bcap, rows, waves, kw, kc, depth, nw = inst
    for N, K in ((301, 4112), (2049, 1040)):
        for B in sorted({bcap, max(1, bcap // 2 + 1)}):
            x, xs, w, ws = case(B, N, K, seed=bcap + rows + N)
            want = expected(x, xs, w, ws)
            plan = tp.PlanI8(N, K, [B])
            for split in (1, 2, 3, 7):
                for stagger in (0, 1):
                    for wpc in (1, 2):
                        plan.set_tactic(B, tp.Tactic(tp.KERNEL_I8_PIPE, bcap, split, rows, waves,
                                                     wpc, kc, depth, kw, nw, stagger))
                        got = run(plan, x, xs, w, ws)
                        assert torch.equal(got.view(torch.int16), want.view(torch.int16)), \
                            (inst, N, K, B, split, stagger, wpc)
            plan.close()
    say(f"[i8 instance {inst}] every split and order bit for bit")


def test_extreme_codes_at_the_longest_sum():
    # every product 2^14 and K as long as it may be: the sum fills the int32
    N, K = 3, tp._binding.MAX_I8_K
    x = torch.full((2, K), -128, dtype=torch.int8)
    x[1] = 127
    w = torch.full((N, K), -128, dtype=torch.int8)
    w[1] = 127
    w[2, ::2] = 127
    xs, ws = torch.tensor([1.0, 0.5]), torch.tensor([1.0, 2.0, 0.25])
    plan = tp.PlanI8(N, K, [2])
    same("i8 extreme", run(plan, x, xs, w, ws), expected(x, xs, w, ws))


def test_scales_of_nan_zero_and_infinity():
    N, K, B = 40, 64, 5
    x, xs, w, ws = case(B, N, K, seed=9)
    x[2] = 0
    xs[2], xs[3], xs[4] = float("nan"), 0.0, float("inf")
    got = run(tp.PlanI8(N, K, [8]), x, xs, w, ws)
    want = expected(x, xs, w, ws)
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and bool(torch.isnan(got[2]).all())
    ok = ~torch.isnan(want)
    assert torch.equal(got[ok], want[ok])


def test_graph_replays_and_alternating_streams():
    N, K, B = 2000, 2048, 100
    plan = tp.PlanI8(N, K, [B])
    x, xs, w, ws = (t.to(DEV) for t in case(B, N, K, seed=2))
    x2 = torch.flip(x, (0,)).contiguous()
    want, want2 = plan.run(x, xs, w, ws), plan.run(x2, xs, w, ws)
    torch.cuda.synchronize()
    xin, y = x.clone(), torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.run(xin, xs, w, ws, y)
    for i in range(4):
        xin.copy_(x2 if i % 2 else x)
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want2 if i % 2 else want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y.zero_()
    torch.cuda.synchronize()
    plan.run(x2, xs, w, ws, y, stream=side)
    side.synchronize()
    assert torch.equal(y, want2)


def test_codes_feed_the_product():
    # rows and weights coded by quant_rows: the product is within the codes'
    # own error of the BF16 product, |y - x.w| <= K/2 (|x|max ws/2..) summed
    g = torch.Generator().manual_seed(4)
    B, N, K = 19, 515, 2064
    x = torch.randn(B, K, generator=g).to(torch.bfloat16)
    w = (0.02 * torch.randn(N, K, generator=g)).to(torch.bfloat16)
    xc, xs = tp.quant_rows(x.to(DEV))
    wc, ws = tp.quant_rows(w.to(DEV))
    y = tp.PlanI8(N, K, [B]).run(xc, xs, wc, ws).cpu().double()
    want = x.double() @ w.double().t()
    xs, ws = xs.cpu().double(), ws.cpu().double()
    # each factor is off by at most half its scale (and the scales by 2^-22):
    # the sum by (|x|_1 ws + |w|_1 xs) / 2 + K xs ws / 4, then BF16 rounding
    tol = (x.double().abs().sum(1)[:, None] * ws / 2 + w.double().abs().sum(1) * xs[:, None] / 2 +
           K * xs[:, None] * ws / 4) * (1 + 2.0 ** -20) + want.abs() * 2.0 ** -7
    assert bool(((y - want).abs() <= tol).all())
    rms = ((y - want).square().mean() / want.square().mean()).sqrt().item()
    say(f"[codes -> product] relative error {rms:.4f}")
