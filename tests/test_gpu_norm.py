"""GPU tests of proj_rms_norm and proj_quant_rows against 64 bits.

Tolerances.  U32 = 2^-24 and U16 = 2^-8 are half a step of float32 and
bfloat16.  h is one FP32 addition (U32).  The sum of squares is a fixed tree
of at most 4 * 8 + 8 + 16 sequential additions, so its relative error is at
most 57 U32 plus 2 U32 for h, and half of that in rstd, plus 3 for the
division, root and its rounding; p adds one product and y another: 40 U32
together bound y before its rounding, and the scale (with its division).
"""
import pytest
import torch

import tp1_skinny_bf16_amd as tp
from gpu_util import DEV, say
from layer_ref import U16, U32, norm

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    torch.cuda.set_device(DEV)


def inputs(rows, D, res, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, D + pad, generator=g)
    x[:, ::max(1, D // 5)] *= 12.0
    r = None if res is None else (2.0 * torch.randn(rows, D + pad, generator=g)).to(res)
    w = (1.0 + 0.1 * torch.randn(D, generator=g)).to(BF)
    return x.to(BF)[:, :D], w, None if r is None else r[:, :D]


def on_device(t):
    """A device copy that keeps the row stride."""
    if t is None or t.is_contiguous():
        return None if t is None else t.to(DEV)
    pad = torch.full((t.shape[0], t.stride(0)), 7.0, dtype=t.dtype, device=DEV)
    pad[:, :t.shape[1]] = t.to(DEV)
    return pad[:, :t.shape[1]]


def check_codes(label, codes, scale, y):
    """Codes and scales of the exact rows y."""
    c, s = codes.cpu().double(), scale.cpu().double()
    top = y.abs().amax(1)
    want = top / 127.0
    serr = ((s - want).abs() / want.clamp(min=1e-300)).max().item()
    t = y / want[:, None].clamp(min=1e-300)
    cerr = (c - t).abs().max().item()
    say(f"[{label}] scale off {serr:.2e}, code off {cerr - 0.5:.2e} beyond a half")
    assert serr <= 40 * U32
    assert cerr <= 0.5 + 127 * 8 * U32
    assert c.abs().max().item() == 127


@pytest.mark.parametrize("rows,D,res,pad", [
    (1, 8, None, 0), (1, 64, BF, 0), (7, 512, F32, 0), (5, 520, BF, 8), (3, 2048, F32, 16),
    (2, 2056, None, 0), (130, 4096, BF, 0), (3, 4104, F32, 24), (1, 7168, BF, 0),
    (65, 7168, F32, 8), (9, 8200, BF, 0), (4, 16384, F32, 0), (2, 16392, BF, 8), (2, 32768, F32, 0),
    (1001, 72, BF, 0),
])
def test_norm_matches_64_bits(rows, D, res, pad):
    x, w, r = inputs(rows, D, res, seed=rows + D, pad=pad)
    h, y = norm(x, w, r, 1e-5)
    xd, wd = on_device(x), w.to(DEV)
    for form in ("y", "codes", "both"):
        rd = on_device(r)
        out = torch.full((rows, D), 3.0, dtype=BF, device=DEV)
        if form == "y":
            tp.rms_norm(xd, wd, residual=rd, eps=1e-5, out=out)
        else:
            codes, scale = tp.rms_norm_i8(xd, wd, residual=rd, eps=1e-5,
                                          out=out if form == "both" else None)
        torch.cuda.synchronize()
        if form != "codes":
            err = ((out.cpu().double() - y).abs() / y.abs().clamp(min=1e-30)).max().item()
            say(f"[norm {rows}x{D} {res} {form}] y off {err / U16:.4f} half steps")
            assert err <= U16 + 42 * U32
        if form != "y":
            check_codes(f"norm {rows}x{D} {res} {form}", codes, scale, y)
        if r is not None:
            u = U16 if res == BF else U32
            err = ((rd.cpu().double() - h).abs() / h.abs().clamp(min=1e-30)).max().item()
            assert err <= u + (2 * U32 if res == BF else 0)
            if pad:
                assert bool((rd.as_strided((rows, pad), (rd.stride(0), 1),
                                           rd.storage_offset() + D)[:-1] == 7.0).all())


@pytest.mark.parametrize("rows,D,pad", [(1, 8, 0), (3, 512, 8), (64, 12288, 0), (5, 7176, 8),
                                        (300, 64, 0), (2, 32768, 0)])
def test_codes_match_64_bits(rows, D, pad):
    x, _, _ = inputs(rows, D, None, seed=D, pad=pad)
    codes, scale = tp.quant_rows(on_device(x))
    check_codes(f"codes {rows}x{D}", codes, scale, x.double())
    # the largest magnitude and its code are exact, so equal rows have equal codes
    again, s2 = tp.quant_rows(on_device(x))
    assert torch.equal(codes, again) and torch.equal(scale, s2)


def test_rows_of_zeros_infinities_nans_and_tiny_values():
    D = 1032
    x = torch.randn(8, D, generator=torch.Generator().manual_seed(3)).to(BF)
    x[1] = 0.0
    x[2, 17] = float("inf")
    x[3, 1031] = float("nan")
    x[4, 5] = float("-inf")
    x[5] = (x[5].float() * 2.0 ** -126).to(BF)        # 127 / max would overflow
    x[6] = torch.finfo(BF).max
    x[7, :] = 0.0
    x[7, 9] = -1.5
    xd = x.to(DEV)
    codes, scale = tp.quant_rows(xd)
    ones = torch.ones(D, dtype=BF, device=DEV)
    nc, ns = tp.rms_norm_i8(xd, ones)
    y = tp.rms_norm(xd, ones)
    torch.cuda.synchronize()
    codes, scale, nc, ns, y = (t.cpu() for t in (codes, scale, nc, ns, y))
    for c, s in ((codes, scale), (nc, ns)):
        for bad in (2, 3, 4):
            assert bool(torch.isnan(s[bad])) and not c[bad].any()
        assert s[1] == 0.0 and not c[1].any()
        assert c[7, 9] == -127 and c[7].abs().sum() == 127
        assert bool((c[6] == 127).all())
    live = [0, 5, 6, 7]
    check = (codes.double() * scale.double()[:, None])[live] - x.double()[live]
    # half a code, and a scale that may be subnormal (2^-149 a step, 127 steps of it)
    tol = scale.double()[live, None] * (0.5 + 127 * 8 * U32) + 127 * 2.0 ** -149
    assert bool((check.abs() <= tol).all())
    assert not y[1].any() and bool(torch.isnan(y[3]).all())
    assert bool(torch.isnan(y[2, 17])) and bool((y[2, :17] == 0).all())


def test_norm_on_a_side_stream_and_in_a_graph():
    x, w, r = inputs(33, 7168, F32, seed=5)
    xd, wd, r0 = x.to(DEV), w.to(DEV), r.to(DEV)
    rd = r0.clone()
    want_c, want_s = tp.rms_norm_i8(xd, wd, residual=rd)
    want_r = rd.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    rd.copy_(r0)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        c, s = tp.rms_norm_i8(xd, wd, residual=rd)
    side.synchronize()
    assert torch.equal(c, want_c) and torch.equal(s, want_s) and torch.equal(rd, want_r)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tp.rms_norm_i8(xd, wd, residual=rd, codes=c, scale=s)
    for _ in range(3):
        rd.copy_(r0)
        c.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c, want_c) and torch.equal(s, want_s) and torch.equal(rd, want_r)


def test_row_offsets_past_32_bits():
    # 300000 rows of 8192: the last rows start past 2^31 elements of x
    rows, D = 300000, 8192
    x = torch.zeros((rows, D), dtype=BF, device=DEV)
    last = torch.randn(D, device=DEV).to(BF)
    x[-1] = last
    codes, scale = tp.quant_rows(x)
    one, s1 = tp.quant_rows(last[None])
    assert torch.equal(codes[-1:], one) and torch.equal(scale[-1:], s1)
    assert not codes[:4].any() and not codes[-5:-1].any()


def test_a_row_of_zeros_without_eps():
    x = torch.ones(3, 256, dtype=torch.bfloat16, device=DEV)
    x[1] = 0
    w = torch.ones(256, dtype=torch.bfloat16, device=DEV)
    out = torch.empty_like(x)
    codes, scale = tp.rms_norm_i8(x, w, eps=0.0, out=out)
    torch.cuda.synchronize()
    assert bool(out[1].isnan().all()) and bool(scale[1].isnan()) and not codes[1].any()
    assert bool((out[::2] == 1).all()) and bool((codes[::2] == 127).all())
