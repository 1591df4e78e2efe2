"""GPU tests of the gated delta rule, recurrent and chunked, against 64 bits.

Tolerances.  With |k| = 1 and beta <= 1 a token's update contracts the state,
so the errors of the tokens add.  The recurrent form holds everything in
FP32: a token's decay is off by a few steps (expf, log1pf: 4 U32 of their
values, times the state), and each inner product sums 128 terms (at most 140
U32 of |S||k|).  With M the largest column norm of the states plus the
largest |v|, a token adds at most 256 U32 * M, and n tokens 256 n U32 * M;
outputs add that (|q| <= 1 after scaling) and half a BF16 step.
The chunked form holds what reaches the state to 2^-23 of each value (and
the output's operands to 2^-11 of their largest); errors of that kind are
independent from element to element, so over the tokens a state remembers
(about 64 of these gates) its relative error in the 2-norm is at most
8 * 2^-23 = 2^-20.
"""
import pytest
import torch

import tp1_skinny_bf16_amd as tp
from gpu_util import DEV, say
from layer_ref import HEAD, U16, U32, columns, delta, delta_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    torch.cuda.set_device(DEV)


def to_device(c):
    return {n: t.to(DEV) if isinstance(t, torch.Tensor) else t for n, t in c.items()}


def check(label, c, seqs, out, state, tokens, **kw):
    q, k, v, b = columns(c)
    want_o, want_s = delta(q, k, v, c["f"], b, c["a_log"], c["dt_bias"], c["state"], seqs, **kw)
    M = max(want_s.norm(dim=2).max().item(), c["state"].double().norm(dim=2).max().item()) + \
        v.double().abs().max().item()
    tol = 256 * max(1, tokens) * U32 * M
    ds = (state.cpu().double() - want_s).abs()
    rel = ((state.cpu().double() - want_s).norm() / want_s.norm()).item()
    do = (out.cpu().double() - want_o).abs() - U16 * want_o.abs()
    say(f"[{label}] state off {ds.max().item():.2e} of {tol:.2e} (rel {rel:.1e}), out "
        f"{do.max().item():.2e}")
    assert bool(torch.isfinite(state).all()) and bool(torch.isfinite(out.float()).all())
    assert ds.max().item() <= tol
    assert rel <= 2.0 ** -20
    assert do.max().item() <= tol
    return want_o, want_s


@pytest.mark.parametrize("requests,tokens,heads,qk,gate", [
    (1, 1, 1, 1, False), (1, 1, 96, 96, False), (3, 2, 12, 6, True), (5, 1, 8, 2, False),
    (7, 4, 6, 6, True), (2, 9, 4, 4, False), (16, 1, 40, 20, True), (12, 3, 96, 48, False),
])
def test_step_matches_64_bits(requests, tokens, heads, qk, gate):
    pool = requests + 2
    c = delta_inputs(requests * tokens, heads, qk, gate, pool, seed=requests + 10 * heads)
    slots = torch.randperm(pool, generator=torch.Generator().manual_seed(1))[:requests].int()
    d = to_device(c)
    q, k, v, b = columns(d)
    out = tp.delta_step(q, k, v, d["f"], b, d["a_log"], d["dt_bias"], d["state"], slots.to(DEV),
                        tokens=tokens)
    torch.cuda.synchronize()
    seqs = [(i * tokens, tokens, int(s)) for i, s in enumerate(slots)]
    check(f"step {requests}x{tokens} H={heads}/{qk} gate={gate}", c, seqs, out, d["state"], tokens)


def test_step_without_norm_and_with_a_scale():
    c = delta_inputs(6, 4, 4, False, 6, seed=8)
    c["row"] *= 0.05          # |k| well under 1
    d = to_device(c)
    q, k, v, b = columns(d)
    out = tp.delta_step(q, k, v, d["f"], b, d["a_log"], d["dt_bias"], d["state"],
                        torch.arange(6, dtype=torch.int32, device=DEV), scale=0.7, l2norm=False)
    check("step raw", c, [(i, 1, i) for i in range(6)], out, d["state"], 1, scale=0.7,
          l2norm=False)


def test_step_padding_and_bad_slots():
    heads, tokens = 8, 2
    c = delta_inputs(12, heads, heads, False, 5, seed=11)
    c["row"][6:8] = float("nan")      # the padded rows hold nothing
    c["f"][6:8] = float("nan")
    slots = torch.tensor([4, 0, 2, -1, 5, 2 ** 30], dtype=torch.int32)   # 5, 2^30: outside
    d = to_device(c)
    q, k, v, b = columns(d)
    out = torch.full((12, heads, HEAD), 5.0, dtype=torch.bfloat16, device=DEV)
    tp.delta_step(q, k, v, d["f"], b, d["a_log"], d["dt_bias"], d["state"], slots.to(DEV),
                  tokens=tokens, out=out)
    torch.cuda.synchronize()
    assert not out[6:].any()
    c["row"][6:8] = 0
    c["f"][6:8] = 0
    check("step padded", c, [(0, 2, 4), (2, 2, 0), (4, 2, 2)], out, d["state"], 2)
    for s in (1, 3):
        assert torch.equal(d["state"][s].cpu(), c["state"][s])


def test_step_takes_requests_of_one_slot_in_order():
    tokens, heads = 2, 5
    c = delta_inputs(12, heads, heads, False, 4, seed=12)
    slots = torch.tensor([3, 1, 3, 0, 1, 3], dtype=torch.int32)
    d = to_device(c)
    q, k, v, b = columns(d)
    out = tp.delta_step(q, k, v, d["f"], b, d["a_log"], d["dt_bias"], d["state"], slots.to(DEV),
                        tokens=tokens)
    seqs = [(i * tokens, tokens, int(s)) for i, s in enumerate(slots)]
    check("step shared slots", c, seqs, out, d["state"], 3 * tokens)


def test_step_extreme_gates():
    # f of -inf keeps the state, +inf clears it; b of +-inf is beta 1 and 0
    c = delta_inputs(4, 2, 2, False, 4, seed=13)
    inf = float("inf")
    c["f"][0], c["f"][1] = -inf, inf
    c["f"][2, :, ::2] = inf
    o = (2 * 2 + 2) * HEAD
    c["row"][2, o], c["row"][3, o] = inf, -inf
    d = to_device(c)
    q, k, v, b = columns(d)
    out = tp.delta_step(q, k, v, d["f"], b, d["a_log"], d["dt_bias"], d["state"],
                        torch.arange(4, dtype=torch.int32, device=DEV))
    check("step extreme gates", c, [(i, 1, i) for i in range(4)], out, d["state"], 1)


def test_step_in_a_graph_follows_new_inputs():
    c = delta_inputs(5, 16, 16, False, 6, seed=14)
    d = to_device(c)
    q, k, v, b = columns(d)
    slots = torch.tensor([5, 0, 1, 2, 3], dtype=torch.int32, device=DEV)
    state, out = d["state"].clone(), torch.zeros(5, 16, HEAD, dtype=torch.bfloat16, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tp.delta_step(q, k, v, d["f"], b, d["a_log"], d["dt_bias"], d["state"], slots, out=out)
    d["state"].copy_(state)
    for i in range(4):
        want = tp.delta_step(q, k, v, d["f"], b, d["a_log"], d["dt_bias"], state, slots)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(state, d["state"])
        slots.copy_(torch.roll(slots, 1))
        d["row"].mul_(-1)


# ---------------------------------------------------------------- sequences

def run_plan(c, lens, slots, **kw):
    d = to_device(c)
    q, k, v, b = columns(d)
    plan = tp.DeltaPlan(lens, slots, heads=c["heads"], qk_heads=c["qk_heads"],
                        n_slots=c["state"].shape[0])
    out = torch.full((c["row"].shape[0], c["heads"], HEAD), 5.0, dtype=torch.bfloat16, device=DEV)
    plan.run(q, k, v, d["f"], b, d["a_log"], d["dt_bias"], d["state"], out=out, **kw)
    torch.cuda.synchronize()
    seqs, r = [], 0
    for n, s in zip(lens, slots):
        seqs.append((r, n, s))
        r += n
    return seqs, out, d


@pytest.mark.parametrize("lens,heads,qk,gate", [
    ([1], 2, 1, False), ([2, 1], 1, 1, True), ([15], 2, 2, False), ([16], 2, 2, True),
    ([17], 3, 1, False), ([31, 0, 33], 2, 2, False), ([63], 2, 2, False), ([64], 2, 1, True),
    ([65], 2, 2, False), ([127, 128, 129], 2, 2, True), ([200, 3, 1, 64, 100], 4, 2, False),
    ([500], 2, 2, False), ([191, 320], 1, 1, True), ([1, 260], 2, 2, False),
    ([300, 16, 5], 2, 1, True),
])
def test_sequences_match_64_bits(lens, heads, qk, gate):
    c = delta_inputs(sum(lens), heads, qk, gate, len(lens) + 1, seed=sum(lens) + heads)
    slots = list(range(len(lens), 0, -1))
    seqs, out, d = run_plan(c, lens, slots)
    check(f"sequences {lens} H={heads}/{qk} gate={gate}", c, seqs, out, d["state"], max(lens))
    assert torch.equal(d["state"][0].cpu(), c["state"][0])


def test_sequences_without_norm_run_row_by_row():
    lens = [90, 0, 3]
    c = delta_inputs(sum(lens), 4, 2, False, 4, seed=20)
    c["row"] *= 0.05          # |k| well under 1
    seqs, out, d = run_plan(c, lens, [2, 1, 3], scale=0.7, l2norm=False)
    check("sequences raw", c, seqs, out, d["state"], 90, scale=0.7, l2norm=False)


def test_sequences_leave_rows_behind_the_last_one():
    lens, extra = [70, 5], 9
    c = delta_inputs(sum(lens) + extra, 2, 2, False, 2, seed=21)
    c["row"][sum(lens):] = float("nan")
    seqs, out, d = run_plan(c, lens, [1, 0])
    assert bool((out[sum(lens):] == 5.0).all())
    c["row"], c["f"] = c["row"][:sum(lens)], c["f"][:sum(lens)]
    check("rows behind", c, seqs, out[:sum(lens)], d["state"], 70)


def test_a_prompt_in_pieces_continues_its_state():
    total, heads = 300, 3
    c = delta_inputs(total, heads, heads, False, 1, seed=22)
    d = to_device(c)
    q, k, v, b = columns(d)
    outs, r = [], 0
    for n in (64, 1, 100, 7, 128):
        plan = tp.DeltaPlan([n], [0], heads=heads, n_slots=1)
        at = slice(r, r + n)
        outs.append(plan.run(q[at], k[at], v[at], d["f"][at], b[at], d["a_log"], d["dt_bias"],
                             d["state"]))
        r += n
    check("prompt in pieces", c, [(0, total, 0)], torch.cat(outs), d["state"], total)


@pytest.mark.parametrize("lens,heads,gate", [([4000], 48, False), ([1500, 40, 1700, 900], 40, True),
                                             ([130] * 40, 24, False), ([6500], 24, True),
                                             ([4500, 20, 1400], 48, False),
                                             ([2100, 2100, 300], 96, False)])
def test_many_chunks_against_the_recurrent_form(lens, heads, gate):
    # many chunks and heads, the last three in several segments with 16, 32 and
    # 64 columns a workgroup; the recurrent form holds
    # everything in FP32 and is itself checked against 64 bits above
    c = delta_inputs(sum(lens), heads, heads, gate, len(lens), seed=31)
    seqs, out, d = run_plan(c, lens, list(range(len(lens))))
    e = to_device(c)
    q, k, v, b = columns(e)
    want = torch.empty_like(out)
    for r0, n, slot in seqs:
        which = torch.tensor([slot], dtype=torch.int32, device=DEV)
        for r in range(r0, r0 + n, 500):
            at = slice(r, min(r + 500, r0 + n))
            want[at] = tp.delta_step(q[at], k[at], v[at], e["f"][at], b[at], e["a_log"],
                                     e["dt_bias"], e["state"], which, tokens=at.stop - r)
    torch.cuda.synchronize()
    rel = ((d["state"] - e["state"]).norm() / e["state"].norm()).item()
    diff = (out.double() - want.double()).norm().item() / want.double().norm().item()
    say(f"[{len(lens)} sequences, {sum(lens)} rows, H={heads}] states differ by {rel:.1e}, "
        f"outputs by {diff:.1e}")
    # both within 2^-20 of 64 bits; outputs differ where one rounds up and the
    # other down: at most a BF16 step (2 U16), on a part of the values
    assert rel <= 2.0 ** -19
    assert diff <= U16


def test_sequences_extreme_gates():
    # tokens that clear the state, keep it, or do so in some channels, at the
    # edges of chunks and in a row
    n = 150
    c = delta_inputs(n, 2, 2, False, 1, seed=23)
    inf = float("inf")
    c["f"][0:3], c["f"][63], c["f"][64], c["f"][100] = -inf, inf, inf, 30.0
    c["f"][80:120, :, ::3] = inf
    c["f"][15:18, :, 5] = inf
    o = (2 * 2 + 2) * HEAD
    c["row"][20, o], c["row"][21, o + 1] = inf, -inf
    seqs, out, d = run_plan(c, [n], [0])
    check("sequences extreme gates", c, seqs, out, d["state"], n)


@pytest.mark.parametrize("head_gate", [False, True])
@pytest.mark.parametrize("heavy,every,at", [(35.0, 16, 0), (70.0, 16, 0), (74.0, 16, 7),
                                            (90.0, 16, 0), (90.0, 16, 9), (40.0, 5, 2),
                                            (60.0, 1, 0), (8.0, 1, 0)])
def test_sequences_of_heavy_finite_gates(heavy, every, at, head_gate):
    # tokens that decay the state by e^-heavy among mild ones: the tokens after
    # them still weigh against each other by ratios near 1
    n = 200
    c = delta_inputs(n, 2, 2, head_gate, 1, seed=27)
    c["a_log"][:] = 0.0
    c["f"][at::every] = heavy
    seqs, out, d = run_plan(c, [n], [0])
    check(f"heavy gates {heavy}/{every}", c, seqs, out, d["state"], n)


def test_sequences_of_repeated_keys_without_decay():
    # the worst case of the triangular inverse: one key over and over, beta 1
    n = 130
    c = delta_inputs(n, 1, 1, False, 1, seed=24)
    c["f"][:] = -40.0
    c["row"][:, HEAD:2 * HEAD] = c["row"][0, HEAD:2 * HEAD]
    c["row"][:, 3 * HEAD] = 20.0
    seqs, out, d = run_plan(c, [n], [0])
    check("repeated keys", c, seqs, out, d["state"], n)


def test_sequences_in_a_graph_and_on_a_side_stream():
    lens, heads = [90, 40], 4
    c = delta_inputs(sum(lens), heads, 2, True, 3, seed=25)
    d = to_device(c)
    q, k, v, b = columns(d)
    plan = tp.DeltaPlan(lens, [2, 0], heads=heads, qk_heads=2, n_slots=3)
    state, out = d["state"].clone(), torch.zeros(sum(lens), heads, HEAD, dtype=torch.bfloat16,
                                                 device=DEV)
    args = (q, k, v, d["f"], b, d["a_log"], d["dt_bias"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.run(*args, d["state"], out=out)
    d["state"].copy_(state)
    for _ in range(3):
        want = plan.run(*args, state)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(state, d["state"])
        d["row"].mul_(-1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want = plan.run(*args, state)
    torch.cuda.synchronize()
    got = plan.run(*args, d["state"], stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(state, d["state"])


def test_the_forms_agree():
    # a sequence token by token through delta_step and at once through a plan
    n, heads = 140, 4
    c = delta_inputs(n, heads, heads, True, 1, seed=26)
    seqs, out, d = run_plan(c, [n], [0])
    e = to_device(c)
    q, k, v, b = columns(e)
    slot = torch.zeros(1, dtype=torch.int32, device=DEV)
    outs = [tp.delta_step(q[t:t + 1], k[t:t + 1], v[t:t + 1], e["f"][t:t + 1], b[t:t + 1],
                          e["a_log"], e["dt_bias"], e["state"], slot) for t in range(n)]
    check("token by token", c, seqs, torch.cat(outs), e["state"], n)
    rel = ((e["state"] - d["state"]).norm() / e["state"].norm()).item()
    say(f"[forms] states differ by {rel:.1e}")
    assert rel <= 2e-5
