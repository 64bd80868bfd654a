"""The training operators where their arithmetic, their waits and their callers
are at an edge: cancelling sums, infinities, time-outs, tensors that autograd
watches, batches split over ranks.

Tolerances are rounding counts, as in test_gpu_training.py: u = 2^-24 is half
a step of fp32, 2^-8 of bf16.  A sum in tensor memory does not round to
nearest: each of its steps is off by at most a whole step, 2 u.
"""

import os
import subprocess
import sys
import textwrap

import numpy as np
import pytest
import torch

import oracle
from mixture_experts_layer_51_b200 import moe as M

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
DEV = "cuda"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# Experts in each layout of dz's bf16 terms (one, two and three 64-wide
# blocks), at the ends of each.
LAYOUTS = [2, 21, 22, 42, 43, 64]


def np64(t):
    return t.detach().double().cpu().numpy()


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def _one_gate(g, T, E):
    """Router inputs in which dz is dgate at one expert a token and zero at
    the others, exactly: a gate of one, scores of zero."""
    idx = torch.randint(0, E, (T, 1), generator=g, device=DEV).int()
    return dict(idx=idx, gate=torch.ones((T, 1), device=DEV), dgate=_randn(g, T, 1),
                scores=torch.zeros((E, T), device=DEV), gating="softmax_topk")


# ------------------------------------------------------------- cancelling sums
@pytest.mark.parametrize("E", LAYOUTS)
def test_dx_keeps_dz_to_24_bits(E):
    """dx_acc cancels dz W_g^T down to its rounding, so that what is left
    shows how many bits of dz the product held."""
    T, d = 600, 136
    g = _gen(E)
    a = _one_gate(g, T, E)
    Wg = _randn(g, d, E, dtype=torch.bfloat16)
    x = _randn(g, T, d, dtype=torch.bfloat16)
    part = a["dgate"].double() * Wg.double().t()[a["idx"][:, 0].long()]
    acc = (-part).to(torch.bfloat16)
    got = M.moe_route_backward(x, Wg, dx_acc=acc, **a)
    want = np64(acc) + np64(part)
    # three products (exact) in two additions, dx_acc in a third, the output
    tol = (2 * 2 + 1 + 1) * U32 * np.abs(np64(part)) + 2.0 ** -8 * np.abs(want)
    err = np.abs(np64(got["dx"]) - want)
    assert np.all(err <= tol), (err / tol).max()


# ---------------------------------------------------------------- masks, waits
@pytest.mark.parametrize("E", [8, 30, 64])
@pytest.mark.parametrize("outputs", [("dx",), ("dx", "dbias")])
def test_dx_of_a_padded_batch_without_dwg(E, outputs):
    """Many tiles a range, with nobody to zero x for: the bits of the whole
    call, and no wait that ran out."""
    T, d = 20000, 2056
    g = _gen(E)
    a = _one_gate(g, T, E)
    a.update(mask=torch.rand(T, generator=g, device=DEV) > 0.3,
             dx_acc=_randn(g, T, d, dtype=torch.bfloat16))
    x, Wg = (_randn(g, *s, dtype=torch.bfloat16) for s in ((T, d), (d, E)))
    want = M.moe_route_backward(x, Wg, **a)
    need = M.moe_route_backward_workspace_bytes(T, d, E, torch.bfloat16)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    for _ in range(5):
        got = M.moe_route_backward(x, Wg, outputs=outputs, ws=ws, **a)
        assert int(ws[:4].view(torch.int32)) == 0
        for name in outputs:
            assert torch.equal(got[name], want[name]), name


# ------------------------------------------------------------------ infinities
# Tokens and type: the one-launch kernel, the tensor cores, fp32 products.
PATHS = [(40, torch.bfloat16), (300, torch.bfloat16), (300, torch.float32)]
PIDS = ["small", "tensor", "fp32"]
INF, NAN = float("inf"), float("nan")


def _same_kind(got, want):
    """NaN where the formula gives NaN, infinities of its signs where it gives
    those, and finite values elsewhere."""
    got = np64(got)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    odd = np.isinf(want)
    assert np.array_equal(got[odd], want[odd])
    assert np.isfinite(got[np.isfinite(want)]).all()


@pytest.mark.parametrize("T,dtype", PATHS, ids=PIDS)
@pytest.mark.parametrize("E", LAYOUTS)
def test_infinities_give_what_fp32_products_give(E, T, dtype):
    """Infinities and NaN in x and W_g at counted tokens, with a gradient at
    every expert: those of the formula, and the other elements keep their
    bits."""
    d = 72
    g = _gen(T + E)
    z = _randn(g, T, E)
    p = torch.softmax(z, 1)
    idx = torch.topk(z, 2, 1).indices.int().contiguous()
    a = dict(idx=idx, gate=p.gather(1, idx.long()).contiguous(), dgate=_randn(g, T, 2),
             scores=p.t().contiguous(), gating="softmax_topk")
    x, Wg = _randn(g, T, d, dtype=dtype), _randn(g, d, E, dtype=dtype)
    plain = M.moe_route_backward(x, Wg, **a)
    dz = oracle.router_dlogits(T, E, idx.cpu().numpy(), np64(a["gate"]), np64(a["dgate"]),
                               np64(a["scores"]), gating="softmax_topk")
    x[5, 3], x[9, 7], x[11, 20], x[12, 20], x[30, 71], x[31, 64] = INF, -INF, INF, -INF, NAN, INF
    Wg[4, 0], Wg[6, 1], Wg[8, 0], Wg[8, 1], Wg[70, E - 1], Wg[71, 0] = INF, -INF, INF, -INF, NAN, INF
    # With two experts and both taken dz may come out as zero or of either
    # sign; the formula's own is what counts only where it is no rounding.
    clear = np.abs(dz) > 1e-5 * np.abs(dz).max()
    rows = [5, 9, 11, 12, 30, 31]
    with np.errstate(invalid="ignore"):
        dx, dWg, _ = oracle.route_backward(np64(x), np64(Wg), dz)
    got = M.moe_route_backward(x, Wg, **a)
    use = clear[rows].all(0)  # experts whose dz at those tokens has a sure sign
    _same_kind(got["dWg"][:, torch.from_numpy(use)], dWg[:, use])
    sure = clear.all(1)
    assert use.any() and sure.any()
    _same_kind(got["dx"][torch.from_numpy(sure)], dx[sure])
    cols = torch.ones(d, dtype=torch.bool)
    cols[[3, 7, 20, 71, 64]] = False
    assert torch.equal(got["dWg"][cols], plain["dWg"][cols])
    cols[:] = True
    cols[[4, 6, 8, 70, 71]] = False
    assert torch.equal(got["dx"][:, cols], plain["dx"][:, cols])


@pytest.mark.parametrize("T,dtype", PATHS, ids=PIDS)
@pytest.mark.parametrize("E", LAYOUTS)
@pytest.mark.parametrize("v", [0.5, -1.0, 1.0 + 2.0 ** -23, 3e38, 1e-20, -1e-33, 1e-36, 1e-39, INF])
def test_an_infinity_times_one_gradient(v, E, T, dtype):
    """One expert of one token has a gradient, of few bits, many, or next to
    the ends of the range: inf times it is inf, times the zeros NaN."""
    d = 64
    g = _gen(E)
    x, Wg = _randn(g, T, d, dtype=dtype), _randn(g, d, E, dtype=dtype)
    a = dict(idx=torch.full((T, 1), E // 2, device=DEV).int(), gate=torch.zeros((T, 1), device=DEV),
             dgate=torch.zeros((T, 1), device=DEV), scores=torch.zeros((E, T), device=DEV),
             gating="softmax_topk")
    a["gate"][7], a["dgate"][7] = 1.0, v
    x[7, 9], Wg[33, E // 2] = -INF, INF
    got = M.moe_route_backward(x, Wg, **a, outputs=("dx", "dWg"))
    # An infinite gate gradient is NaN at every expert of the token already:
    # dz_e = [e = idx] g dg - p_e sum g dg, and p_e = 0 times infinity is NaN.
    sign = NAN if v == INF else 1.0 if v > 0 else -1.0
    want = np.full(E, NAN)
    want[E // 2] = -sign * INF
    assert np.array_equal(np64(got["dWg"][9]), want, equal_nan=True)
    assert np.array_equal(np64(got["dx"][7, 33]), sign * INF, equal_nan=True)
    assert got["dx"][8, 33].isnan()


@pytest.mark.parametrize("T,dtype", PATHS, ids=PIDS)
@pytest.mark.parametrize("E", LAYOUTS)
@pytest.mark.parametrize("v", [1.0, 1.0 + 2.0 ** -23, 3.0e38, 3.4e38, -3.4e38, 1e-29, 1e-31, 1e-39,
                               INF, -INF, NAN])
def test_a_gradient_at_the_ends_of_the_range(v, E, T, dtype):
    """As far as dz itself goes, in every layout of its terms: three terms of
    one sign hold every value down to 2^-100, and the smaller ones to three
    times bf16's least value."""
    d = 64
    x = torch.zeros((T, d), dtype=dtype, device=DEV)
    x[7, 3] = 1.0
    Wg = torch.zeros((d, E), dtype=dtype, device=DEV)
    Wg[:, E - 1] = 0.5
    a = dict(idx=torch.full((T, 1), E - 1, device=DEV).int(), gate=torch.zeros((T, 1), device=DEV),
             dgate=torch.zeros((T, 1), device=DEV), scores=torch.zeros((E, T), device=DEV),
             gating="softmax_topk")
    a["gate"][7], a["dgate"][7] = 1.0, v
    got = M.moe_route_backward(x, Wg, **a)
    dx, dWg = np64(got["dx"]), np64(got["dWg"])
    v = float(a["dgate"][7])  # in fp32
    if not np.isfinite(v):  # p_e = 0 times the sum of g dg, infinite or NaN, is NaN
        assert np.isnan(dWg[3]).all() and np.isnan(dx[7]).all()
        return
    # two additions, each off by at most a step; the least terms
    tol = 4 * U32 * abs(v) + 3 * 2.0 ** -133
    assert abs(dWg[3, E - 1] - v) <= tol and abs(float(got["dbias"][E - 1]) - v) <= 2.0 ** -149
    # half the smallest numbers of the output's type more
    u = torch.finfo(dtype).eps / 2
    assert np.all(np.abs(dx[7] - v / 2) <= tol + u * abs(v) / 2 + 2.0 ** -134)
    assert not np.delete(dx, 7, 0).any()


@pytest.mark.parametrize("T,dtype", PATHS, ids=PIDS)
@pytest.mark.parametrize("E", LAYOUTS)
def test_an_infinite_gradient_of_the_loss(E, T, dtype):
    """dz of both infinities at one token: each expert's in dW_g, NaN in the
    sums over the experts (infinities of both signs)."""
    d = 64
    g = _gen(T * E)
    scores = torch.zeros((E, T), device=DEV)
    scores[:, 7] = torch.softmax(_randn(g, E), 0)
    counts = torch.zeros(E, dtype=torch.int32, device=DEV)
    counts[0] = T  # f = (1, 0, ...): f_e - sum f p is 1 - p_0 at the first expert, else -p_0
    x, Wg = _randn(g, T, d, dtype=dtype), torch.ones((d, E), dtype=dtype, device=DEV)
    x[7] = x[7].abs() + 1
    tokens = torch.tensor([T], dtype=torch.int32, device=DEV)
    mask = torch.arange(T, device=DEV) == 7  # the other tokens' p of 0 times infinity is NaN
    got = M.moe_route_backward(x, Wg, torch.zeros((T, 1), dtype=torch.int32, device=DEV),
                               scores=scores, counts=counts, tokens=tokens, coef=1.0,
                               dloss=torch.tensor([INF], device=DEV), mask=mask)
    want = np.full(E, -INF)
    want[0] = INF
    assert np.array_equal(np64(got["dWg"]), np.broadcast_to(want, (d, E)))
    assert np.array_equal(np64(got["dbias"]), want)
    dx = np64(got["dx"])
    assert np.isnan(dx[7]).all() and not np.delete(dx, 7, 0).any()


# ------------------------------------------------------- waits that run out
STALLED = textwrap.dedent("""
    import sys, torch
    sys.path.insert(0, {root!r})
    from mixture_experts_layer_51_b200 import moe as M
    ERR_TIMEOUT_MMA = 1 << 1
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")
    # T, d, E, whether a launch of its own adds the ranges, mask, outputs
    CASES = [(600, 200, 8, False, False, ("dx", "dWg", "dbias")),
             (2000, 392, 64, False, True, ("dx", "dWg", "dbias")),
             (20000, 136, 30, True, True, ("dx", "dWg", "dbias")),
             (900, 264, 30, False, True, ("dx",)),
             (700, 264, 43, False, False, ("dx", "dbias")),
             (700, 264, 43, False, True, ("dWg",))]
    calls = []
    for T, d, E, _, masked, outputs in CASES:
        p = torch.softmax(rand(T, E), 1)
        idx = torch.topk(p, 2, 1).indices.int().contiguous()
        need = M.moe_route_backward_workspace_bytes(T, d, E, torch.bfloat16)
        calls.append(dict(
            x=rand(T, d).bfloat16(), Wg=rand(d, E).bfloat16(), idx=idx,
            gate=p.gather(1, idx.long()).contiguous(), dgate=rand(T, 2),
            scores=p.t().contiguous(), gating="softmax_topk", outputs=outputs,
            mask=torch.arange(T, device="cuda") % 3 > 0 if masked else None,
            dx_acc=rand(T, d).bfloat16() if "dx" in outputs else None,
            ws=torch.empty(need, dtype=torch.uint8, device="cuda")))
    bads, words = [], []
    for a in calls:  # the launches that stall, dx in place
        buf = a["dx_acc"].clone() if a["dx_acc"] is not None else None
        bads.append(M.moe_route_backward(**dict(a, dx_acc=buf, dx=buf)))
        words.append(int(a["ws"][:4].view(torch.int32)))
    for (T, d, E, many, _, outputs), a, bad, word in zip(CASES, calls, bads, words):
        assert word & ERR_TIMEOUT_MMA, word
        good = M.moe_route_backward(**a)
        assert int(a["ws"][:4].view(torch.int32)) == 0
        assert all(torch.isfinite(good[n].float()).all() for n in outputs)
        if "dx" in outputs:
            lost = bad["dx"].isnan()
            rows = int(lost.any(1).sum())
            assert 0 < rows and (rows == T or rows % 128 == 0), rows
            assert lost[:rows, :128].all() and not lost[rows:].any() and not lost[:, 128:].any()
            assert torch.equal(bad["dx"][~lost], good["dx"][~lost])
        if "dWg" in outputs:
            lost = bad["dWg"].isnan()
            assert lost[:128].all()
            assert lost[128:].all() if many else not lost[128:].any()
            assert torch.equal(bad["dWg"][~lost], good["dWg"][~lost])
        if "dbias" in outputs:
            assert torch.equal(bad["dbias"], good["dbias"])
        print("REPORTED")
""")


def test_a_wait_that_runs_out_marks_what_it_left():
    """One CTA of the tensor-core kernel runs out of its bounded waits: the
    error word says so, its block of dx and its columns of dW_g are NaN, the
    rest is right, and so is the next call of the same."""
    env = dict(os.environ, MOE_DEBUG_STALL_ROUTE="6")
    r = subprocess.run([sys.executable, "-c", STALLED.format(root=ROOT)], env=env,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr[-3000:]
    assert r.stdout.count("REPORTED") == 6


def test_a_step_keeps_the_router_error_word():
    from mixture_experts_layer_51_b200.workloads import Workload, make_inputs
    w = Workload("t", T=300, d=64, E=4, k=2, H=64, act="swiglu", dtype="bf16", cf=0.0, seed=9)
    t = make_inputs(w, DEV)
    layer = M.MoELayer(t["Wg"], t["bias"], t["W1"], t["W3"], t["W2"], w.k, w.cf, w.act)
    for x in (t["x"], t["x"][:7], t["x"][:0]):
        y, _, step = layer.forward_train(x, coef=0.1)
        layer.backward_combine(step, torch.ones_like(y))
        layer.backward_router(step)
        assert step["router_error"].dtype == torch.int32 and int(step["router_error"]) == 0


# ------------------------------------------------------- the residual in place
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T,d,k", [(4000, 64, 2), (3001, 128, 4), (2000, 2056, 2), (300, 4104, 8),
                                   (1, 136, 1)])
def test_the_combine_onto_its_residual_again_and_again(T, d, k, dtype):
    """y is the residual, call after call with nothing in between: the bits of
    the same calls into buffers of their own."""
    g = _gen(T + d + k)
    rows = T * k
    o = _randn(g, rows, d, dtype=dtype)
    pos = torch.randperm(rows, generator=g, device=DEV).int().view(T, k)
    gate = torch.rand((T, k), generator=g, device=DEV)
    rng = torch.tensor([11, 12], device=DEV)
    start = _randn(g, T, d, dtype=dtype)
    buf, want = start.clone(), start
    for _ in range(6):
        M.moe_combine_dropout(o, pos, gate, 0.3, rng, residual=buf, y=buf)
    for _ in range(6):
        want = M.moe_combine_dropout(o, pos, gate, 0.3, rng, residual=want)
    assert torch.equal(buf, want)


# ------------------------------------------------------------------- autograd
def test_calls_refuse_tensors_that_autograd_watches():
    """Every entry point, for any of its tensors; under no_grad they run."""
    from mixture_experts_layer_51_b200.workloads import Workload, make_inputs
    w = Workload("t", T=300, d=64, E=4, k=2, H=64, act="swiglu", dtype="bf16", cf=0.0, seed=9)
    t = make_inputs(w, DEV)
    layer = M.MoELayer(t["Wg"], t["bias"], t["W1"], t["W3"], t["W2"], w.k, w.cf, w.act)
    x = t["x"]
    y, _, s = layer.forward_train(x, coef=0.1)
    watched = x.clone().requires_grad_()
    o, gate, scores = (s[n].clone().requires_grad_() for n in ("o", "gate", "scores"))
    calls = [
        lambda: layer.forward_train(watched),
        lambda: layer.forward_train(watched * 1),
        lambda: layer.forward_train(x, residual=watched),
        lambda: layer.backward_combine(s, watched),
        lambda: M.moe_balance_loss(scores, s["idx"], 0.1)["loss"],
        lambda: M.moe_combine_dropout(o, s["pos"], s["gate"]),
        lambda: M.moe_combine_dropout(s["o"], s["pos"], gate),
        lambda: M.moe_combine_dropout_backward(y, o, s["pos"], s["gate"]),
        lambda: M.moe_route_backward(watched, layer.Wg, s["idx"], s["gate"], s["gate"]),
        lambda: M.moe_route_backward(x, layer.Wg, s["idx"], s["gate"], gate),
    ]
    for call in calls:
        with pytest.raises(ValueError, match="requires a gradient"):
            call()
        with torch.no_grad():
            call()


# ---------------------------------------------------- a batch split over ranks
@pytest.mark.parametrize("T,d,E,k,dtype", [(1500, 136, 8, 2, torch.bfloat16),
                                           (3001, 264, 64, 8, torch.bfloat16),
                                           (1100, 72, 12, 3, torch.float32)])
def test_two_parts_of_a_batch_with_summed_counts(T, d, E, k, dtype):
    """counts, tokens and prob_sum of two parts add up to the whole batch's;
    with the sums each part's dx is the whole's, bit for bit, and dW_g and
    dbias add up to it."""
    g = _gen(T)
    z = _randn(g, T, E) + _randn(g, E)
    scores, idx = torch.softmax(z, 1), torch.topk(z, k, 1).indices.int().contiguous()
    x, Wg = _randn(g, T, d, dtype=dtype), _randn(g, d, E, dtype=dtype)
    mask = torch.rand(T, generator=g, device=DEV) > 0.2
    dloss = torch.tensor([float(T)], device=DEV)
    parts = [slice(0, 2 * T // 5), slice(2 * T // 5, T)]

    def balance(rows):
        return M.moe_balance_loss(scores[rows].t().contiguous(), idx[rows], 0.2, mask=mask[rows])

    def backward(rows, counts, tokens):
        return M.moe_route_backward(x[rows], Wg, idx[rows], scores=scores[rows].t().contiguous(),
                                    counts=counts, tokens=tokens, coef=0.2, dloss=dloss,
                                    mask=mask[rows])
    whole = balance(slice(0, T))
    some = [balance(r) for r in parts]
    sums = {n: some[0][n] + some[1][n] for n in ("counts", "tokens", "prob_sum")}
    assert torch.equal(sums["counts"], whole["counts"])
    assert torch.equal(sums["tokens"], whole["tokens"])
    n = int(sums["tokens"])
    loss = 0.2 * E * float((np64(sums["counts"]) / (n * k) * np64(sums["prob_sum"]) / n).sum())
    assert abs(float(whole["loss"]) - loss) <= (2 * T + 4) * U32 * loss
    want = backward(slice(0, T), whole["counts"], whole["tokens"])
    got = [backward(r, sums["counts"], sums["tokens"]) for r in parts]
    assert torch.equal(torch.cat([got[0]["dx"], got[1]["dx"]]), want["dx"])
    dz = oracle.router_dlogits(T, E, idx=idx.cpu().numpy(), scores=np64(scores.t()),
                               counts=np64(whole["counts"]), tokens=n, coef=0.2,
                               dloss=float(T), mask=mask.cpu().numpy())
    f = np64(whole["counts"]) / (n * k)
    # dz by a difference of two sums, then T terms each way, the parts' sum
    size = np.abs(dz) + 0.2 * E * np64(scores) * np.abs(np64(scores) @ f)[:, None] * 2
    ax = np.abs(np64(x)) * mask.cpu().numpy()[:, None]
    for name, tol in (("dWg", ax.T @ size), ("dbias", size.sum(0))):
        err = np.abs(np64(got[0][name]) + np64(got[1][name]) - np64(want[name]))
        assert np.all(err <= 2 * (T + E + 12) * U32 * tol), name


# ----------------------------------------- one expert, nothing but padding
BOTH = [torch.bfloat16, torch.float32]


@pytest.mark.parametrize("dtype", BOTH, ids=["tensor", "fp32"])
@pytest.mark.parametrize("gating", ["topk_softmax", "softmax_topk"])
def test_one_expert_past_the_small_batches(gating, dtype):
    """A router with one expert has nothing to learn: zeros, and dx_acc."""
    T, d = 700, 136
    g = _gen(1)
    acc = _randn(g, T, d, dtype=dtype)
    one = torch.ones((T, 1), device=DEV)
    got = M.moe_route_backward(_randn(g, T, d, dtype=dtype), _randn(g, d, 1, dtype=dtype),
                               torch.zeros((T, 1), device=DEV).int(), one, _randn(g, T, 1),
                               one.t().contiguous(), torch.tensor([T], device=DEV).int(),
                               torch.tensor([T], device=DEV).int(), coef=0.5, gating=gating,
                               dx_acc=acc)
    assert torch.equal(got["dx"], acc) and not got["dWg"].any() and not got["dbias"].any()


@pytest.mark.parametrize("dtype", BOTH, ids=["tensor", "fp32"])
@pytest.mark.parametrize("E", [8, 30, 64])
def test_a_batch_of_padding_past_the_small_batches(E, dtype):
    """The mask leaves no token: zeros and dx_acc, whatever the rest holds."""
    T, d, k = 900, 264, 2
    g = _gen(E)
    mask = torch.zeros(T, dtype=torch.bool, device=DEV)
    nan = lambda *s: torch.full(s, NAN, device=DEV)  # noqa: E731
    idx = torch.full((T, k), 1 << 30, device=DEV).int()
    bal = M.moe_balance_loss(nan(E, T), idx, 0.5, mask=mask)
    assert float(bal["loss"]) == 0 and int(bal["tokens"]) == 0 and not bal["prob_sum"].any()
    acc = _randn(g, T, d, dtype=dtype)
    got = M.moe_route_backward(nan(T, d).to(dtype), _randn(g, d, E, dtype=dtype), idx, nan(T, k),
                               nan(T, k), nan(E, T), bal["counts"], bal["tokens"], coef=0.5,
                               mask=mask, gating="softmax_topk", dx_acc=acc)
    assert torch.equal(got["dx"], acc) and not got["dWg"].any() and not got["dbias"].any()


# ------------------------------------------ around the choice of who adds dW_g
@pytest.mark.parametrize("T,d,E,dtype", [
    (3400, 1024, 8, "fp32"), (3700, 1024, 8, "fp32"),    # by the bytes of x
    (6800, 1024, 8, "bf16"), (7400, 1024, 8, "bf16"),
    (1001, 1032, 40, "fp32"), (1001, 1032, 41, "fp32"),  # by the products
    (1650, 1032, 64, "bf16"), (1700, 1032, 64, "bf16")])
def test_route_backward_around_the_summing_launch(T, d, E, dtype):
    from test_gpu_training import _check_route, _route_case
    a = _route_case(T, d, E, 2, dtype, "softmax_topk", 1.0, True, True, "some", True)
    got, again = M.moe_route_backward(**a), M.moe_route_backward(**a)
    _check_route(a, got)
    assert all(torch.equal(got[n], again[n]) for n in got)


# --------------------------------------------------- rows narrower than a tile
@pytest.mark.parametrize("E", [8, 30, 64])
@pytest.mark.parametrize("d", [8, 24, 56, 72])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_route_backward_of_narrow_rows_past_the_small_batches(d, E, dtype):
    from test_gpu_training import _check_route, _route_case
    a = _route_case(1100, d, E, 2, dtype, "softmax_topk", 1.0, True, True, "some", True)
    whole = [torch.full((1100 * d + 128,), 7, dtype=a["x"].dtype, device=DEV),
             torch.full((d * E + 128,), 7.0, device=DEV)]
    got = M.moe_route_backward(**a, dx=whole[0][64:-64].view(1100, d),
                               dWg=whole[1][64:-64].view(d, E))
    _check_route(a, got)
    assert all((w[:64] == 7).all() and (w[-64:] == 7).all() for w in whole)


# ----------------------------------------------- elements past 2^31, bytes 2^32
def _philox(first, count, seed, offset):
    """The 16-bit lanes of counters first .. first + count - 1 (Salmon et al.)."""
    u32, u64 = np.uint32, np.uint64
    n = np.arange(first, first + count, dtype=u64)
    ctr = [n.astype(u32), (n >> u64(32)).astype(u32), np.full(n.shape, offset, u32),
           np.zeros(n.shape, u32)]
    key = [seed, 0]
    for _ in range(10):
        lo, hi = ctr[0].astype(u64) * u64(0xD2511F53), ctr[2].astype(u64) * u64(0xCD9E8D57)
        ctr = [(hi >> u64(32)).astype(u32) ^ ctr[1] ^ u32(key[0]), hi.astype(u32),
               (lo >> u64(32)).astype(u32) ^ ctr[3] ^ u32(key[1]), lo.astype(u32)]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    return np.ascontiguousarray(np.stack(ctr, 1)).view(np.uint16)


def test_offsets_past_32_bits():
    """The last rows of tensors of more than 2^31 elements, against calls on
    copies of those rows."""
    T, d, E, k, n = 560000, 4096, 8, 2, 700  # 2.3 G elements, 4.6 GB
    g = _gen(8)
    big = torch.empty((T, d), dtype=torch.bfloat16, device=DEV)
    for t in range(0, T, 40000):
        big[t:t + 40000] = _randn(g, min(40000, T - t), d, dtype=torch.bfloat16)
    tail = slice(T - n, T)
    # combine: every slot's row is one of the last n of o
    pos = (T - n + torch.randperm(n, generator=g, device=DEV)).int().view(n // k, k)
    gate = torch.rand((n // k, k), generator=g, device=DEV)
    rng = torch.tensor([3, 4], device=DEV)
    part = big[tail].clone()
    near = (pos - (T - n)).contiguous()
    y = M.moe_combine_dropout(big, pos, gate, 0.1, rng)
    assert torch.equal(y, M.moe_combine_dropout(part, near, gate, 0.1, rng))
    dy = _randn(g, n // k, d, dtype=torch.bfloat16)
    d_o = torch.zeros_like(big)
    d_o, dgate = M.moe_combine_dropout_backward(dy, big, pos, gate, 0.1, rng, d_o=d_o)
    want_o, want_g = M.moe_combine_dropout_backward(dy, part, near, gate, 0.1, rng)
    assert torch.equal(d_o[tail], want_o) and torch.equal(dgate, want_g)
    assert not d_o[:n].any()
    # as many tokens: the generator's counter and y's rows
    pos = torch.full((T, 1), -1, device=DEV).int()
    pos[tail] = torch.arange(n, device=DEV).int()[:, None]
    one = torch.ones((T, 1), device=DEV)
    y = M.moe_combine_dropout(part, pos, one, 0.25, rng, y=d_o)
    # element c of token t: counter (t d + c) / 8, here past 2^28
    words = _philox((T - n) * d // 8, n * d // 8, 3, 4)
    kept = torch.from_numpy(words.reshape(n, d) >= oracle.dropout_threshold(0.25)).to(DEV)
    scaled = (part.float() * (65536 / (65536 - oracle.dropout_threshold(0.25)))).bfloat16()
    assert torch.equal(y[tail], torch.where(kept, scaled, 0))
    del y
    # router: the last tokens' dx, and dW_g of a gradient at those tokens alone
    idx = torch.randint(0, E, (T, 1), generator=g, device=DEV).int()
    dgate = torch.zeros((T, 1), device=DEV)
    dgate[tail] = _randn(g, n, 1)
    zero = torch.zeros((E, T), device=DEV)
    Wg = _randn(g, d, E, dtype=torch.bfloat16)
    got = M.moe_route_backward(big, Wg, idx, one, dgate, zero, gating="softmax_topk", dx=d_o)
    a = dict(idx=idx[tail].contiguous(), gate=one[tail].contiguous(),
             dgate=dgate[tail].contiguous(), scores=zero[:, tail].contiguous(),
             gating="softmax_topk")
    want = M.moe_route_backward(part, Wg, **a)
    assert torch.equal(got["dx"][tail], want["dx"]) and not got["dx"][:n].any()
    size = np64(part.abs()).T @ (np.eye(E)[a["idx"][:, 0].cpu().numpy()] * np.abs(np64(a["dgate"])))
    assert np.all(np.abs(np64(got["dWg"]) - np64(want["dWg"])) <= 2 * (n + 8) * U32 * size)
