"""CPU tests of the layer operators' argument checks (no launch happens: every
call is refused, is empty, or uses a host-only plan)."""
import ctypes

import pytest
import torch

import tp1_skinny_bf16_amd as tp
from tp1_skinny_bf16_amd import _binding as bd

X, R, W, Y, C, S = (0x100000 * i for i in range(1, 7))     # never dereferenced


def norm(rows=4, D=64, x=X, ldx=0, res=None, ldr=0, wide=0, w=W, eps=1e-6, y=Y, c=None, s=None):
    return tp.library().proj_rms_norm(rows, D, x, ldx, res, ldr, wide, w, eps, y, c, s, None)


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(D=0), dict(D=60), dict(D=32776), dict(ldx=56), dict(x=None), dict(w=None),
    dict(y=None), dict(c=C), dict(s=S), dict(y=None, s=S), dict(wide=2, res=R),
    dict(res=R, ldr=32), dict(eps=-1.0), dict(eps=float("nan")),
    dict(y=X), dict(y=X + 256), dict(res=X), dict(y=R, res=R), dict(y=W), dict(c=Y, s=S),
    dict(c=C, s=C + 16), dict(res=Y + 128),
])
def test_norm_refuses(kw):
    assert norm(**kw) == tp.PROJ_EINVAL


@pytest.mark.parametrize("kw", [
    dict(x=X + 8), dict(w=W + 2), dict(y=Y + 8), dict(res=R + 8), dict(c=C + 4, s=S),
    dict(c=C, s=S + 2), dict(ldx=68), dict(res=R, ldr=68),
])
def test_norm_refuses_misaligned(kw):
    assert norm(**kw) == tp.PROJ_EALIGN


def test_norm_of_no_rows_is_nothing():
    assert norm(rows=0, x=None, w=None, y=None) == tp.PROJ_OK
    assert tp.library().proj_quant_rows(0, 64, None, 0, None, None, None) == tp.PROJ_OK


def test_quant_refuses():
    q = tp.library().proj_quant_rows
    assert q(4, 64, X, 0, None, S, None) == tp.PROJ_EINVAL
    assert q(4, 64, X, 0, C, None, None) == tp.PROJ_EINVAL
    assert q(4, 12, X, 0, C, S, None) == tp.PROJ_EINVAL
    assert q(4, 64, X, 32, C, S, None) == tp.PROJ_EINVAL
    assert q(4, 64, X, 0, X + 8, S, None) == tp.PROJ_EINVAL
    assert q(4, 64, X, 0, C, C + 64, None) == tp.PROJ_EINVAL
    assert q(4, 64, X + 2, 0, C, S, None) == tp.PROJ_EALIGN
    assert q(4, 64, X, 0, C + 1, S, None) == tp.PROJ_EALIGN


@pytest.mark.parametrize("N,K,batches", [
    (0, 64, [1]), (64, 0, [1]), (64, 24, [1]), (64, 131072, [1]), (64, 64, []), (64, 64, [2, 2]),
    (64, 64, [257]), (64, -16, [1])])
def test_i8_plan_refuses(N, K, batches):
    with pytest.raises(tp.ProjError) as e:
        tp.PlanI8(N, K, batches, host_only=True)
    assert e.value.code == tp.PROJ_EINVAL


def test_i8_run_refuses():
    p = tp.PlanI8(128, 256, [1, 8], host_only=True)
    XS, WS = C, S
    run = p.run_ptr
    assert run(0, 0, 0, 0, 0, 0, 0) == tp.PROJ_OK
    assert run(9, X, 0, XS, W, WS, Y) == tp.PROJ_EBATCH
    assert run(-1, X, 0, XS, W, WS, Y) == tp.PROJ_EBATCH
    assert run(8, X, 240, XS, W, WS, Y) == tp.PROJ_EINVAL
    assert run(8, X, 264, XS, W, WS, Y) == tp.PROJ_EALIGN
    assert run(8, X + 8, 0, XS, W, WS, Y) == tp.PROJ_EALIGN
    assert run(8, X, 0, XS, W, WS, Y + 2) == tp.PROJ_EALIGN
    for bad in ((None, XS, W, WS, Y), (X, None, W, WS, Y), (X, XS, None, WS, Y),
                (X, XS, W, None, Y), (X, XS, W, WS, None), (X, XS, W, WS, X), (X, XS, W, WS, W),
                (X, Y + 16, W, WS, Y), (X, XS, W, Y + 64, Y)):
        assert run(8, bad[0], 0, *bad[1:]) == tp.PROJ_EINVAL
    assert run(8, X, 0, XS, W, WS, Y) == tp.PROJ_ENODEV


def test_every_i8_bin_has_a_valid_tactic():
    for N, K in [(14560, 7168), (49376, 7168), (7168, 12288), (1820, 7168), (33, 16), (1, 64),
                 (5, 131056), (100000, 160)]:
        p = tp.PlanI8(N, K, [1, 2, 4, 8, 16, 32, 64, 128, 256], host_only=True)
        for b in range(1, 257):
            t, bin_ = p.tactic(b)
            assert t.kernel == tp.KERNEL_I8_PIPE and t.bcap >= bin_ >= b
            p.set_tactic(bin_, t)
        assert p.workspace_bytes < 1 << 30
        with pytest.raises(tp.ProjError):
            p.set_tactic(16, tp.Tactic(tp.KERNEL_MFMA_PIPE, 16, 1, 4, 1, 1, 256, 3, 2, 8))
        with pytest.raises(tp.ProjError):
            p.set_tactic(3, p.tactic(4)[0])


def io(heads=4, qk=2, **kw):
    base = dict(q=0x1000000, k=0x2000000, v=0x3000000, f=0x4000000, b=0x5000000, ldq=0, ldk=0,
                ldv=0, ldf=0, ldb=0, a_log=0x6000000, dt_bias=0x7000000, state=0x10000000,
                out=0x8000000, ldo=0, scale=1.0, l2norm=1, head_gate=0)
    base.update(kw)
    return bd.DeltaIO(*[base[n] for n, _ in bd.DeltaIO._fields_])


def step(heads=4, qk=2, requests=3, tokens=2, slots=0x9000000, n_slots=8, **kw):
    return tp.library().proj_delta_step(ctypes.byref(io(heads, qk, **kw)), heads, qk, requests,
                                        tokens, slots, n_slots, None)


@pytest.mark.parametrize("kw", [
    dict(heads=0), dict(heads=1025, qk=1025), dict(qk=3), dict(qk=0), dict(requests=-1),
    dict(requests=4097), dict(tokens=0), dict(tokens=1025), dict(n_slots=0), dict(slots=None),
    dict(q=None), dict(state=None), dict(out=None), dict(a_log=None), dict(dt_bias=None),
    dict(head_gate=2), dict(ldq=128), dict(ldv=256), dict(ldf=256), dict(ldb=2), dict(ldo=8),
    dict(out=0x3000000), dict(out=0x10000000), dict(state=0x1000000 - 64), dict(out=0x9000000 - 64),
    dict(slots=0x10000000),
])
def test_delta_step_refuses(kw):
    assert step(**kw) == tp.PROJ_EINVAL


@pytest.mark.parametrize("kw", [
    dict(q=0x1000008), dict(k=0x2000002), dict(v=0x3000008), dict(state=0x10000008),
    dict(out=0x8000008), dict(ldq=260), dict(ldv=516), dict(ldf=516), dict(f=0x4000008),
    dict(b=0x5000001), dict(slots=0x9000002), dict(ldo=516),
])
def test_delta_step_refuses_misaligned(kw):
    assert step(**kw) == tp.PROJ_EALIGN


def test_delta_step_of_no_requests_is_nothing():
    assert step(requests=0, slots=None, q=None) == tp.PROJ_OK


@pytest.mark.parametrize("kw", [
    dict(lens=[3, -1]), dict(slots=[0, 0]), dict(slots=[0, 5]), dict(slots=[-1, 1]),
    dict(heads=0), dict(heads=3, qk_heads=2), dict(n_slots=0), dict(lens=[], slots=[]),
    dict(lens=[1 << 28, 1]),
])
def test_delta_plan_refuses(kw):
    args = dict(lens=[3, 4], slots=[0, 1], heads=4, qk_heads=2, n_slots=5)
    args.update(kw)
    with pytest.raises(tp.ProjError) as e:
        tp.DeltaPlan(args.pop("lens"), args.pop("slots"), host_only=True, **args)
    assert e.value.code == tp.PROJ_EINVAL


def test_delta_run_refuses():
    p = tp.DeltaPlan([3, 0, 4], [2, 0, 1], heads=4, qk_heads=2, n_slots=8, host_only=True)
    assert p.rows == 7
    run = lambda **kw: tp.library().proj_delta_run(p._h, ctypes.byref(io(**kw)), None)  # noqa: E731
    assert run() == tp.PROJ_ENODEV
    assert run(v=None) == tp.PROJ_EINVAL
    assert run(out=0x2000000) == tp.PROJ_EINVAL
    assert run(k=0x2000004) == tp.PROJ_EALIGN
    assert tp.library().proj_delta_run(None, ctypes.byref(io()), None) == tp.PROJ_EINVAL
    empty = tp.DeltaPlan([0], [0], heads=4, qk_heads=2, n_slots=8, host_only=True)
    assert tp.library().proj_delta_run(empty._h, ctypes.byref(io(q=None)), None) == tp.PROJ_OK


def test_bindings_refuse_host_and_mistyped_tensors():
    bf, f32 = torch.bfloat16, torch.float32
    x, w = torch.zeros(2, 64, dtype=bf), torch.zeros(64, dtype=bf)
    with pytest.raises(TypeError):
        tp.rms_norm(x.float(), w)
    with pytest.raises(TypeError):
        tp.rms_norm(x, w.float())
    with pytest.raises(ValueError):
        tp.rms_norm(x, w[:32])
    with pytest.raises(ValueError):
        tp.rms_norm(x.t(), w)
    with pytest.raises(TypeError):
        tp.quant_rows(x, codes=torch.zeros(2, 64))
    with pytest.raises(ValueError):
        tp.quant_rows(x, scale=torch.zeros(3))
    with pytest.raises(ValueError):          # host tensors
        tp.rms_norm(x, w)
    with pytest.raises(ValueError):
        tp.quant_rows(x)
    p = tp.PlanI8(8, 64, [2], host_only=True)
    c, s = torch.zeros(2, 64, dtype=torch.int8), torch.zeros(2)
    wc, ws = torch.zeros(8, 64, dtype=torch.int8), torch.zeros(8)
    with pytest.raises(ValueError):          # host tensors
        p.run(c, s, wc, ws)
    with pytest.raises(TypeError):
        p.run(c, s.double(), wc, ws)
    with pytest.raises(ValueError):
        p.run(c, s[:1], wc, ws)
    with pytest.raises(ValueError):
        p.run(c[:, :32], s, wc, ws)
    t = dict(q=torch.zeros(2, 2, 128, dtype=bf), k=torch.zeros(2, 2, 128, dtype=bf),
             v=torch.zeros(2, 4, 128, dtype=bf), f=torch.zeros(2, 4, dtype=bf),
             b=torch.zeros(2, 4, dtype=bf), a_log=torch.zeros(4), dt_bias=torch.zeros(4),
             state=torch.zeros(3, 4, 128, 128), slots=torch.zeros(2, dtype=torch.int32))
    for name, bad in (("q", t["q"].float()), ("slots", t["slots"].long()), ("f", t["f"].float()),
                      ("a_log", t["a_log"].to(bf)), ("state", t["state"].to(bf))):
        with pytest.raises(TypeError):
            tp.delta_step(**{**t, name: bad})
    for name, bad in (("q", t["q"][:1]), ("k", t["k"][:, :1]), ("v", t["v"][:, :3]),
                      ("f", torch.zeros(2, 4, 64, dtype=bf)), ("dt_bias", torch.zeros(4, 128)),
                      ("state", t["state"][:, :2]), ("slots", t["slots"][:1]),
                      ("out", torch.zeros(2, 3, 128, dtype=bf))):
        with pytest.raises(ValueError):
            tp.delta_step(**{**t, name: bad})
    with pytest.raises(ValueError):          # host tensors
        tp.delta_step(**t)
    plan = tp.DeltaPlan([2], [0], heads=4, qk_heads=2, n_slots=3, host_only=True)
    t.pop("slots")
    with pytest.raises(ValueError):
        plan.run(**{**t, "state": torch.zeros(4, 4, 128, 128)})
    with pytest.raises(ValueError):
        tp.DeltaPlan([2, 1], [0], heads=4, n_slots=3, host_only=True)


def test_bindings_refuse_rows_that_overlap():
    # expanded rows have stride 0, which the C calls read as contiguous
    bf = torch.bfloat16
    x = torch.zeros(1, 64, dtype=bf).expand(3, 64)
    full, w = torch.zeros(3, 64, dtype=bf), torch.zeros(64, dtype=bf)
    half = torch.zeros(256, dtype=bf).as_strided((3, 64), (32, 1))
    for bad in (x, half):
        for call in (lambda: tp.rms_norm(bad, w), lambda: tp.rms_norm_i8(bad, w),
                     lambda: tp.quant_rows(bad), lambda: tp.rms_norm(full, w, residual=bad)):
            with pytest.raises(ValueError, match="overlap"):
                call()
    p = tp.PlanI8(64, 64, [4], host_only=True)
    c, s = torch.zeros(1, 64, dtype=torch.int8).expand(3, 64), torch.zeros(3)
    with pytest.raises(ValueError, match="overlap"):
        p.run(c, s, torch.zeros(64, 64, dtype=torch.int8), torch.zeros(64))
    t = dict(q=torch.zeros(2, 2, 128, dtype=bf), k=torch.zeros(2, 2, 128, dtype=bf),
             v=torch.zeros(2, 4, 128, dtype=bf), f=torch.zeros(2, 4, dtype=bf),
             b=torch.zeros(2, 4, dtype=bf), a_log=torch.zeros(4), dt_bias=torch.zeros(4),
             state=torch.zeros(3, 4, 128, 128), slots=torch.zeros(2, dtype=torch.int32))
    for name in ("q", "k", "v", "f", "b"):
        with pytest.raises(ValueError, match="overlap"):
            tp.delta_step(**{**t, name: t[name][:1].expand(t[name].shape)})
    with pytest.raises(ValueError, match="overlap"):
        tp.delta_step(**t, out=torch.zeros(1, 4, 128, dtype=bf).expand(2, 4, 128))
