"""The training operators against the fp64 oracle: the balance loss, the
combine with dropout, and the backward passes of the combine and the router.

Tolerances are rounding counts.  u = 2^-24 is half a step of fp32; a sum of n
terms, in whatever order, is off by at most n u sum |terms| (first order); an
output rounded to bf16 by 2^-8 |value| more, to fp32 by 2^-24 |value|.
"""

import numpy as np
import pytest
import torch

import oracle
from mixture_experts_layer_51_b200 import moe as M

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
DEV = "cuda"


def _u(dtype):
    return torch.finfo(dtype).eps / 2


def np64(t):
    return t.detach().double().cpu().numpy()


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def _selection(g, T, E, k, skew=1.0):
    """Scores [E, T] and distinct experts [T, k] by descending score."""
    z = _randn(g, T, E) + skew * _randn(g, E)
    p = torch.softmax(z, 1)
    idx = torch.topk(z, k, 1).indices.int().contiguous()
    return p.t().contiguous(), idx


def _mask(g, T, kind):
    if kind is None:
        return None
    m = torch.rand(T, generator=g, device=DEV) > 0.3
    if kind == "none":
        m[:] = False
    if kind == "tail":
        m[:] = torch.arange(T, device=DEV) < T // 3
    return m if kind != "bytes" else m.to(torch.uint8)


# ------------------------------------------------------------- balance loss
@pytest.mark.parametrize("T,E,k,mask", [
    (0, 8, 2, None), (1, 1, 1, None), (1, 64, 8, "some"), (31, 5, 2, "some"), (32, 8, 8, None),
    (33, 7, 3, "bytes"), (255, 4, 1, None), (256, 64, 8, "some"), (257, 33, 5, "none"),
    (1000, 8, 2, None), (4097, 64, 8, "some"), (70001, 63, 6, "some"), (131072, 2, 1, None),
    (300000, 16, 4, "bytes")])
def test_balance_loss(T, E, k, mask):
    g = _gen(T + 7 * E + k)
    scores, idx = _selection(g, T, E, k)
    m = _mask(g, T, mask)
    coef = 0.37
    got = M.moe_balance_loss(scores, idx, coef, mask=m)
    again = M.moe_balance_loss(scores, idx, coef, mask=m)
    loss, prob_sum, counts, n = oracle.balance_loss(np64(scores), idx.cpu().numpy(), E, coef,
                                                    None if m is None else m.cpu().numpy())
    assert got["counts"].tolist() == counts.tolist() and got["tokens"].tolist() == [n]
    # at most n additions of nonnegative terms, each of them at most the sum
    tol = max(n, 1) * U32
    assert np.all(np.abs(np64(got["prob_sum"]) - prob_sum) <= tol * prob_sum)
    assert abs(float(got["loss"]) - loss) <= (tol + 2 * U32) * abs(loss)
    for name in got:
        assert torch.equal(got[name], again[name]), name


def test_balance_loss_takes_anything_where_the_mask_is_off():
    """NaN and infinite scores and wild indices of padding tokens; indices
    outside the experts are counted nowhere for the others too."""
    g = _gen(3)
    T, E, k = 777, 12, 3
    scores, idx = _selection(g, T, E, k)
    m = _mask(g, T, "some")
    want = M.moe_balance_loss(scores, idx, 0.1, mask=m)
    wild, widx = scores.clone(), idx.clone()
    wild[:, ~m] = float("nan")
    wild[0, ~m] = float("inf")
    widx[~m] = 1 << 30
    got = M.moe_balance_loss(wild, widx, 0.1, mask=m)
    for name in got:
        assert torch.equal(got[name], want[name]), name
    widx = idx.clone()
    widx[5, 0], widx[6, 1] = -1, E
    got = M.moe_balance_loss(scores, widx, 0.1)
    ok = (widx >= 0) & (widx < E)
    assert got["counts"].tolist() == torch.bincount(widx[ok], minlength=E).tolist()


def test_balance_loss_with_one_expert_taking_all():
    T, E = 50000, 64
    scores = torch.full((E, T), 1 / E, device=DEV)
    idx = torch.full((T, 1), 63, dtype=torch.int32, device=DEV)
    got = M.moe_balance_loss(scores, idx, 1.0)
    assert got["counts"].tolist() == [0] * 63 + [T]
    assert abs(float(got["loss"]) - 1.0) <= T * U32


# ---------------------------------------------------------- router backward
ROUTE = [
    # T, d, E, k, dtype, gating, scale, gates, loss, mask, acc
    (1, 64, 2, 1, "fp32", "topk_softmax", 1.0, True, True, None, False),
    (1, 8, 64, 8, "bf16", "softmax_topk", 1.0, True, True, None, True),
    (5, 72, 3, 3, "bf16", "topk_softmax", 2.0, True, False, "some", False),
    (31, 136, 8, 2, "bf16", "topk_softmax", 1.0, True, True, None, True),
    (33, 128, 8, 2, "fp32", "softmax_topk", 4.0, True, True, "some", True),
    (64, 256, 16, 4, "bf16", "softmax_topk", 1.0, True, True, "none", True),
    (127, 200, 17, 4, "bf16", "topk_softmax", 1.0, True, True, "bytes", False),
    (128, 1032, 32, 2, "bf16", "topk_softmax", 1.0, False, True, None, True),
    (129, 64, 64, 8, "fp32", "softmax_topk", 0.5, True, False, None, False),
    (300, 520, 33, 8, "bf16", "softmax_topk", 1.0, True, True, "some", True),
    (1000, 96, 5, 1, "bf16", "softmax_topk", 1.0, True, True, None, False),
    (1000, 1024, 8, 2, "bf16", "topk_softmax", 1.0, True, True, None, True),
    (1027, 264, 64, 8, "bf16", "topk_softmax", 1.0, True, True, "some", False),
    (2500, 392, 48, 6, "fp32", "topk_softmax", 1.0, True, True, "some", True),
    (5000, 64, 12, 2, "bf16", "topk_softmax", 1.0, True, True, None, True),
    (3001, 4104, 9, 2, "bf16", "topk_softmax", 1.0, True, True, "some", False),
    (20000, 72, 64, 8, "bf16", "softmax_topk", 1.0, True, True, "some", True),
    # the widths at which the terms of dz take another block
    (260, 136, 21, 3, "bf16", "softmax_topk", 1.0, True, True, "some", True),
    (260, 136, 22, 3, "bf16", "topk_softmax", 1.0, True, True, None, False),
    (260, 136, 42, 3, "bf16", "softmax_topk", 1.0, True, True, None, True),
    (260, 136, 43, 3, "bf16", "topk_softmax", 1.0, True, True, "some", False),
    (700, 320, 61, 8, "bf16", "softmax_topk", 1.0, True, True, "some", True),
    (700, 320, 63, 7, "fp32", "softmax_topk", 1.0, True, True, "some", True),
    # ranges of many tiles, three blocks of terms
    (6000, 2056, 64, 8, "bf16", "softmax_topk", 1.0, True, True, "some", True),
    # many ranges of few columns, and a large pass, whose ranges a launch adds
    (20000, 64, 44, 2, "bf16", "topk_softmax", 1.0, True, True, "some", False),
    (20000, 64, 8, 2, "fp32", "softmax_topk", 1.0, True, True, "some", True),
    (9000, 520, 30, 2, "bf16", "topk_softmax", 1.0, False, True, None, False),
    (8200, 1160, 6, 2, "bf16", "topk_softmax", 1.0, False, True, None, True),
    (8200, 1032, 50, 3, "fp32", "softmax_topk", 1.0, True, True, "some", True),
    # around the sizes up to which one launch does it all
    (256, 264, 8, 2, "bf16", "softmax_topk", 1.0, True, True, "some", True),
    (256, 264, 16, 4, "fp32", "topk_softmax", 2.0, True, True, "some", True),
    (257, 264, 16, 4, "fp32", "topk_softmax", 2.0, True, True, "some", True),
    (255, 40, 9, 8, "bf16", "topk_softmax", 1.0, True, True, None, False),
    (128, 4736, 32, 2, "bf16", "softmax_topk", 1.0, True, True, "bytes", True),
    (129, 4736, 32, 2, "bf16", "softmax_topk", 1.0, True, True, "bytes", True),
    (64, 104, 64, 8, "bf16", "softmax_topk", 1.0, True, True, "some", False),
    (64, 104, 57, 8, "fp32", "topk_softmax", 1.0, True, True, "tail", True),
    (2, 4744, 3, 1, "bf16", "softmax_topk", 1.0, True, True, None, True),
    # one expert: nothing to learn, zeros
    (70, 72, 1, 1, "bf16", "topk_softmax", 1.0, True, True, "some", True),
    (70, 72, 1, 1, "fp32", "softmax_topk", 1.0, True, True, None, False),
    # more column blocks than SMs: a range of 4, 5 and 9 tiles each
    (512, 19208, 8, 2, "bf16", "topk_softmax", 1.0, True, True, None, True),
    (640, 19208, 64, 2, "bf16", "softmax_topk", 1.0, True, True, "some", False),
    (1025, 19208, 24, 2, "bf16", "topk_softmax", 1.0, True, True, "some", True),
    # a padded batch whose tail is all padding (whole tiles of it)
    (1500, 264, 8, 2, "bf16", "topk_softmax", 1.0, True, True, "tail", True),
]


def _route_case(T, d, E, k, dtype, gating, scale, gates, loss, mask, acc, seed=0):
    g = _gen(T * 31 + d + E + seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    scores, idx = _selection(g, T, E, k)
    m = _mask(g, T, mask)
    sel = scores.t().gather(1, idx.long())
    gate = scale * (sel / sel.sum(1, keepdim=True) if gating == "topk_softmax" else sel)
    a = dict(x=_randn(g, T, d, dtype=dt), Wg=_randn(g, d, E, dtype=dt), idx=idx, scores=scores,
             mask=m, gating=gating, gate_scale=scale, coef=0.0)
    if gates:
        a.update(gate=gate.contiguous(), dgate=_randn(g, T, k))
    if loss:
        bal = M.moe_balance_loss(scores, idx, 0.2, mask=m)
        a.update(counts=bal["counts"], tokens=bal["tokens"], coef=0.2,
                 dloss=torch.rand(1, generator=g, device=DEV) * T)
    if acc:
        a["dx_acc"] = _randn(g, T, d, dtype=dt)
    return a


def _check_route(a, got, outputs=("dx", "dWg", "dbias")):
    x, Wg, idx = a["x"], a["Wg"], a["idx"].cpu().numpy()
    T, d = x.shape
    E, k = Wg.shape[1], idx.shape[1]
    n = lambda t: None if t is None else np64(t)  # noqa: E731
    m = None if a["mask"] is None else a["mask"].cpu().numpy().astype(bool)
    gate, dgate, scores = n(a.get("gate")), n(a.get("dgate")), n(a["scores"])
    counts = None if a.get("counts") is None else a["counts"].cpu().numpy()
    tokens = 0 if counts is None else int(a["tokens"])
    dloss = 1.0 if a.get("dloss") is None else float(a["dloss"])
    dz = oracle.router_dlogits(T, E, idx, gate, dgate, scores, counts, tokens, a["coef"], dloss, m,
                               a["gating"], a["gate_scale"])
    dx, dWg, dbias = oracle.route_backward(np64(x), np64(Wg), dz, n(a.get("dx_acc")), m)
    # How far dz itself may be off: sums of at most E + k terms of these
    # sizes, and a dozen roundings of products, quotients and differences.
    size = np.zeros((T, E))
    if dgate is not None:
        part = np.abs(gate * dgate)
        total = part.sum(1, keepdims=True)
        if a["gating"] == "topk_softmax":
            spread = part + np.abs(gate) * total / a["gate_scale"]
        else:
            spread = part
            size += scores.T * total
        for j in range(k):
            size[np.arange(T), idx[:, j]] += spread[:, j]
    if counts is not None and tokens:
        f = counts / (tokens * k)
        size += abs(dloss * a["coef"]) * E / tokens * scores.T * (f + (scores.T @ f)[:, None])
    if m is not None:
        size[~m] = 0
    edz = (E + k + 12) * U32 * size
    ax, aw = np.abs(np64(x)), np.abs(np64(Wg))
    if m is not None:
        ax = np.where(m[:, None], ax, 0)
    u = _u(x.dtype)
    if "dx" in outputs:
        # a bf16 layer may carry dz in two bf16 terms here: 2^-16 of it
        carry = 2.0 ** -16 if x.dtype == torch.bfloat16 else 0.0
        tol = edz @ aw.T + ((E + 2) * U32 + carry) * (np.abs(dz) @ aw.T) + (u + U32) * np.abs(dx)
        if a.get("dx_acc") is not None:
            tol += 2 * U32 * np.abs(np64(a["dx_acc"]))
        err = np.abs(np64(got["dx"]) - dx)
        assert np.all(err <= tol + 1e-30), (err / (tol + 1e-30)).max()
    if "dWg" in outputs:
        tol = ax.T @ edz + (T + 8) * U32 * (ax.T @ np.abs(dz))
        err = np.abs(np64(got["dWg"]) - dWg)
        assert np.all(err <= tol + 1e-30), (err / (tol + 1e-30)).max()
        # and close in the whole: the errors of fp32 sums do not add up in step
        if np.linalg.norm(dWg) > 0:
            rough = np.linalg.norm(ax.T @ edz) / np.linalg.norm(dWg)
            assert np.linalg.norm(np64(got["dWg"]) - dWg) <= (4e-6 + rough) * np.linalg.norm(dWg)
    if "dbias" in outputs:
        tol = edz.sum(0) + (T + 8) * U32 * np.abs(dz).sum(0)
        err = np.abs(np64(got["dbias"]) - dbias)
        assert np.all(err <= tol + 1e-30), (err / (tol + 1e-30)).max()


@pytest.mark.parametrize("case", ROUTE, ids=lambda c: "x".join(map(str, c[:4])) + "-" + c[4])
def test_route_backward(case):
    a = _route_case(*case)
    got = M.moe_route_backward(**a)
    again = M.moe_route_backward(**a)
    _check_route(a, got)
    for name in got:
        assert torch.equal(got[name], again[name]), name


@pytest.mark.parametrize("outputs", [("dx",), ("dWg",), ("dbias",), ("dx", "dbias"),
                                     ("dWg", "dbias")])
@pytest.mark.parametrize("case", [ROUTE[3], ROUTE[4], ROUTE[12], ROUTE[13], ROUTE[14]],
                         ids=["bf16-small", "fp32-small", "bf16", "fp32", "bf16-many"])
def test_route_backward_of_some_outputs(case, outputs):
    """Asking for less gives the same bits of what is asked for."""
    a = _route_case(*case)
    want = M.moe_route_backward(**a)
    got = M.moe_route_backward(**a, outputs=outputs)
    assert set(got) == set(outputs)
    for name in outputs:
        assert torch.equal(got[name], want[name]), name


@pytest.mark.parametrize("case", [ROUTE[4], ROUTE[6], ROUTE[9], ROUTE[13], ROUTE[15]],
                         ids=["fp32-small", "bf16-small", "bf16", "fp32", "bf16-wide"])
def test_route_backward_never_looks_at_padding(case):
    """NaN in a padding token's x, scores, gates and gate gradients reaches
    nothing; its dx row is its dx_acc, or zero."""
    a = _route_case(*case)
    want = M.moe_route_backward(**a)
    off = ~a["mask"].bool()
    assert off.any()
    b = dict(a, x=a["x"].clone(), scores=a["scores"].clone(), gate=a["gate"].clone(),
             dgate=a["dgate"].clone(), idx=a["idx"].clone())
    b["x"][off] = float("nan")
    b["scores"][:, off] = float("nan")
    b["gate"][off] = float("inf")
    b["dgate"][off] = float("nan")
    b["idx"][off] = -5
    got = M.moe_route_backward(**b)
    for name in got:
        assert torch.equal(got[name], want[name]), name
    rows = a["dx_acc"][off] if a.get("dx_acc") is not None else torch.zeros_like(a["x"][off])
    assert torch.equal(got["dx"][off], rows)


@pytest.mark.parametrize("case", [ROUTE[3], ROUTE[4], ROUTE[13], ROUTE[16]],
                         ids=["bf16-small", "fp32-small", "fp32", "bf16"])
def test_route_backward_adds_in_place(case):
    a = _route_case(*case)
    want = M.moe_route_backward(**a)["dx"]
    buf = a["dx_acc"].clone()
    got = M.moe_route_backward(**dict(a, dx_acc=buf, dx=buf))["dx"]
    assert got.data_ptr() == buf.data_ptr() and torch.equal(got, want)


def test_route_backward_stays_inside_its_buffers():
    """Guard rows around every output and the workspace keep their bytes."""
    for case in (ROUTE[1], ROUTE[2], ROUTE[6], ROUTE[8], ROUTE[9], ROUTE[13], ROUTE[15]):
        a = _route_case(*case)
        T, d = a["x"].shape
        E = a["Wg"].shape[1]
        dt = a["x"].dtype

        def guarded(n, dtype):
            buf = torch.full((n + 128,), 77, dtype=dtype, device=DEV)
            return buf, buf[64:64 + n]
        need = M.moe_route_backward_workspace_bytes(T, d, E, dt)
        bufs = [guarded(T * d, dt), guarded(d * E, torch.float32), guarded(E, torch.float32),
                guarded(need, torch.uint8)]
        got = M.moe_route_backward(**a, dx=bufs[0][1].view(T, d), dWg=bufs[1][1].view(d, E),
                                   dbias=bufs[2][1], ws=bufs[3][1])
        _check_route(a, got)
        for whole, inner in bufs:
            n = inner.numel()
            assert (whole[:64] == 77).all() and (whole[64 + n:] == 77).all()


def test_route_backward_of_an_empty_batch():
    E, d = 6, 64
    z = lambda *s, **k: torch.zeros(s, device=DEV, **k)  # noqa: E731
    got = M.moe_route_backward(z(0, d, dtype=torch.bfloat16), z(d, E, dtype=torch.bfloat16),
                               z(0, 2, dtype=torch.int32), gate=z(0, 2), dgate=z(0, 2),
                               dWg=torch.ones((d, E), device=DEV), dbias=torch.ones(E, device=DEV))
    assert not got["dWg"].any() and not got["dbias"].any() and got["dx"].shape == (0, d)


def test_route_backward_with_the_same_expert_twice_and_none():
    """A token that names one expert twice adds both terms there; an index
    outside the experts adds nothing at its place."""
    a = _route_case(300, 64, 8, 3, "fp32", "topk_softmax", 1.0, True, False, None, False)
    a["idx"][:, 1] = a["idx"][:, 0]
    a["idx"][::7, 2] = 99
    got = M.moe_route_backward(**a)
    dz = oracle.router_dlogits(300, 8, a["idx"].cpu().numpy(), np64(a["gate"]), np64(a["dgate"]))
    _, dWg, dbias = oracle.route_backward(np64(a["x"]), np64(a["Wg"]), dz)
    size = np.abs(np64(a["x"])).T @ np.abs(dz)
    assert np.all(np.abs(np64(got["dWg"]) - dWg) <= (300 + 64) * U32 * 4 * size.max())
    assert np.all(np.abs(np64(got["dbias"]) - dbias) <= (300 + 64) * U32 * 4 * np.abs(dz).sum(0).max())


# ------------------------------------------------------ combine with dropout
def _combine_case(T, d, E, k, dtype, cap=None, seed=0):
    g = _gen(T * 13 + d + k + seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    _, idx = _selection(g, T, E, k)
    rows = M.moe_rows_for_capacity(T, E, k, cap)
    x = torch.zeros((T, d), dtype=dt, device=DEV)
    perm = M.moe_permute(x, idx, E, None, capacity=-1 if cap is None else cap)
    return dict(o=_randn(g, max(rows, 128), d, dtype=dt), pos=perm["pos"],
                gate=torch.rand((T, k), generator=g, device=DEV),
                rng=torch.tensor([0x1234567_89ABCDEF, 5 + (9 << 33)], device=DEV)), g


COMBINE = [
    # T, d, E, k, dtype, p, residual, capacity
    (1, 8, 1, 1, "bf16", 0.5, True, None), (1, 4096, 8, 2, "bf16", 0.1, True, None),
    (3, 4104, 64, 8, "fp32", 0.3, False, None), (7, 264, 5, 2, "fp32", 0.25, True, 2),
    (33, 520, 8, 8, "bf16", 0.9, True, None), (64, 256, 4, 1, "bf16", 0.0, False, 9),
    (255, 1032, 16, 3, "fp32", 0.0, True, 0), (300, 2056, 32, 4, "bf16", 0.99999, True, None),
    (1000, 136, 64, 8, "bf16", 0.1, False, 60), (1300, 1024, 8, 2, "bf16", 1e-6, True, None),
    (2049, 64, 12, 5, "fp32", 0.5, True, None),
    # rows of eight lanes (up to 128 elements), and one element group more
    (1001, 64, 8, 2, "bf16", 0.1, True, None), (45, 72, 7, 3, "fp32", 0.4, True, 20),
    (77, 128, 16, 4, "bf16", 0.1, False, None), (515, 128, 64, 7, "bf16", 0.0, True, 50),
    (31, 8, 3, 1, "fp32", 0.5, True, None), (90, 136, 9, 4, "bf16", 0.2, True, 30),
    # three and four slots, rows of several warps
    (5, 4096, 8, 3, "bf16", 0.1, True, None), (2000, 4104, 8, 4, "bf16", 0.1, True, 700),
    (900, 1544, 6, 4, "fp32", 0.1, False, None),
]
CIDS = ["x".join(map(str, c[:4])) + "-" + c[4] for c in COMBINE]


def _keep(a, p, T, d):
    if oracle.dropout_threshold(p) == 0:
        return None
    seed, offset = (int(v) for v in a["rng"].cpu())
    return oracle.dropout_keep(p, seed, offset, T, d)


@pytest.mark.parametrize("case", COMBINE, ids=CIDS)
def test_combine_dropout(case):
    T, d, E, k, dtype, p, residual, cap = case
    a, g = _combine_case(T, d, E, k, dtype, cap)
    res = _randn(g, T, d, dtype=a["o"].dtype) if residual else None
    y = M.moe_combine_dropout(**a, p=p, residual=res)
    keep = _keep(a, p, T, d)
    o, pos, gate = np64(a["o"]), a["pos"].cpu().numpy(), np64(a["gate"])
    r = None if res is None else np64(res)
    want = oracle.combine_dropout(o, pos, gate, keep, p, r)
    size = oracle.combine_dropout(np.abs(o), pos, np.abs(gate), keep, p)
    # k products and sums, the scale (and its own rounding), the residual
    tol = (k + 3) * U32 * size + 2 * U32 * np.abs(want) + _u(a["o"].dtype) * np.abs(want)
    assert np.all(np.abs(np64(y) - want) <= tol + 1e-30)
    if keep is not None:  # dropped elements are the residual itself, bit for bit
        drop = torch.from_numpy(~keep).to(DEV)
        rest = res if res is not None else torch.zeros_like(y)
        assert torch.equal(y[drop], rest[drop])
    if p == 0 and res is None:
        assert torch.equal(y, M.moe_unpermute_combine(a["o"], a["pos"], a["gate"], a["o"].dtype))
    if res is not None:
        buf = res.clone()
        assert torch.equal(M.moe_combine_dropout(**a, p=p, residual=buf, y=buf), y)
        assert torch.equal(buf, y)


@pytest.mark.parametrize("case", COMBINE, ids=CIDS)
def test_combine_dropout_backward(case):
    T, d, E, k, dtype, p, _, cap = case
    a, g = _combine_case(T, d, E, k, dtype, cap, seed=1)
    dt = a["o"].dtype
    dy = _randn(g, T, d, dtype=dt)
    guard = torch.full_like(a["o"], 3.0)
    d_o, dgate = M.moe_combine_dropout_backward(dy, **a, p=p, d_o=guard.clone())
    again = M.moe_combine_dropout_backward(dy, **a, p=p, d_o=guard.clone())
    assert torch.equal(d_o, again[0]) and torch.equal(dgate, again[1])
    keep = _keep(a, p, T, d)
    o, pos, gate = np64(a["o"]), a["pos"].cpu().numpy(), np64(a["gate"])
    want_o, want_g = oracle.combine_dropout_backward(np64(dy), o, pos, gate, keep, p)
    owned = np.zeros(o.shape[0], bool)
    owned[pos[pos >= 0]] = True
    assert (d_o[torch.from_numpy(~owned).to(DEV)] == 3.0).all()  # left as they were
    # the scale (rounded itself), the product with the gate, the output
    tol = (3 * U32 + _u(dt)) * np.abs(want_o)
    assert np.all((np.abs(np64(d_o) - want_o) <= tol + 1e-30)[owned])
    _, size = oracle.combine_dropout_backward(np.abs(np64(dy)), np.abs(o), pos, gate, keep, p)
    # a lane adds d / 32 products, more where warps share a row, then a tree
    assert np.all(np.abs(np64(dgate) - want_g) <= (d / 16 + 32) * U32 * size + 1e-30)
    assert (dgate[a["pos"] < 0] == 0).all()


def test_a_dropped_element_is_left_out_whatever_stands_there():
    T, d, k, p = 200, 256, 2, 0.4
    a, g = _combine_case(T, d, 8, k, "bf16")
    dy = _randn(g, T, d, dtype=torch.bfloat16)
    keep = torch.from_numpy(_keep(a, p, T, d)).to(DEV)
    y = M.moe_combine_dropout(**a, p=p)
    d_o, dgate = M.moe_combine_dropout_backward(dy, **a, p=p)
    wild, wdy = a["o"].clone(), dy.clone()
    wdy[~keep] = float("nan")
    for j in range(k):
        rows = wild[a["pos"][:, j].long()]
        wild[a["pos"][:, j].long()] = torch.where(keep, rows, float("inf"))
    b = dict(a, o=wild)
    own = a["pos"].long().flatten()
    assert torch.equal(M.moe_combine_dropout(**b, p=p), y)
    got_o, got_g = M.moe_combine_dropout_backward(wdy, **b, p=p)
    assert torch.equal(got_o[own], d_o[own]) and torch.equal(got_g, dgate)


def test_rows_of_dropped_slots_are_not_read():
    """Padding rows and rows nobody owns may hold NaN."""
    a, g = _combine_case(500, 72, 8, 2, "fp32", cap=40)
    dy = _randn(g, 500, 72)
    y = M.moe_combine_dropout(**a)
    d_o, dgate = M.moe_combine_dropout_backward(dy, **a, d_o=torch.zeros_like(a["o"]))
    pos = a["pos"]
    owned = torch.zeros(a["o"].shape[0], dtype=torch.bool, device=DEV)
    owned[pos[pos >= 0].long()] = True
    b = dict(a, o=torch.where(owned[:, None], a["o"], float("nan")), gate=a["gate"].clone())
    b["gate"][pos < 0] = float("nan")
    assert torch.equal(M.moe_combine_dropout(**b), y)
    got = M.moe_combine_dropout_backward(dy, **b, d_o=torch.zeros_like(a["o"]))
    assert torch.equal(got[0], d_o) and torch.equal(got[1], dgate)


# ------------------------------------------------- graphs, streams, the step
def test_a_captured_combine_reads_the_generator_when_it_runs():
    a, g = _combine_case(400, 512, 8, 2, "bf16")
    dy = _randn(g, 400, 512, dtype=torch.bfloat16)
    y = torch.zeros_like(dy)
    d_o, dgate = torch.zeros_like(a["o"]), torch.zeros_like(a["gate"])
    calls = lambda: (M.moe_combine_dropout(**a, p=0.3, y=y),  # noqa: E731
                     M.moe_combine_dropout_backward(dy, **a, p=0.3, d_o=d_o, dgate=dgate))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    seen = []
    for offset in (1, 2, 1):
        a["rng"][1] = offset
        graph.replay()
        seen.append((y.clone(), d_o.clone(), dgate.clone()))
        ey = M.moe_combine_dropout(**a, p=0.3)
        eo, eg = M.moe_combine_dropout_backward(dy, **a, p=0.3, d_o=torch.zeros_like(d_o))
        assert torch.equal(seen[-1][0], ey) and torch.equal(seen[-1][1], eo)
        assert torch.equal(seen[-1][2], eg)
    assert not torch.equal(seen[0][0], seen[1][0])
    assert all(torch.equal(p, q) for p, q in zip(seen[0], seen[2]))


def test_captured_loss_and_router_backward_share_nothing():
    """Two graphs over the same inputs and one workspace each, replayed in
    turn and at once on two streams, give the eager bits."""
    a = _route_case(3000, 256, 32, 4, "bf16", "softmax_topk", 1.0, True, True, None, False)
    want_l = M.moe_balance_loss(a["scores"], a["idx"], 0.2)
    want = M.moe_route_backward(**a)
    graphs, outs = [], []
    for _ in range(2):
        ws = [torch.empty(M.moe_balance_loss_workspace_bytes(3000, 32), dtype=torch.uint8,
                          device=DEV),
              torch.empty(M.moe_route_backward_workspace_bytes(3000, 256, 32, torch.bfloat16),
                          dtype=torch.uint8, device=DEV)]
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            loss = M.moe_balance_loss(a["scores"], a["idx"], 0.2, ws=ws[0])
            back = M.moe_route_backward(**dict(a, counts=loss["counts"], tokens=loss["tokens"]),
                                        ws=ws[1])
        graphs.append((gr, ws))
        outs.append((loss, back))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for (gr, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for loss, back in outs:
        assert all(torch.equal(loss[n], want_l[n]) for n in want_l)
        assert all(torch.equal(back[n], want[n]) for n in want)


def test_calls_on_a_stream_of_their_own():
    """stream=: what is allocated inside belongs to that stream."""
    a = _route_case(2000, 512, 16, 2, "bf16", "topk_softmax", 1.0, True, True, "some", True)
    c, g = _combine_case(2000, 512, 16, 2, "bf16")
    want = M.moe_route_backward(**a)
    y = M.moe_combine_dropout(**c, p=0.2)
    bal = M.moe_balance_loss(a["scores"], a["idx"], 0.2, mask=a["mask"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        got = M.moe_route_backward(**a, stream=s)
        got_y = M.moe_combine_dropout(**c, p=0.2, stream=s)
        got_b = M.moe_balance_loss(a["scores"], a["idx"], 0.2, mask=a["mask"], stream=s)
        torch.empty(1 << 22, device=DEV).fill_(float("nan"))  # reuses freed memory, if any
    s.synchronize()
    assert all(torch.equal(got[n], want[n]) for n in want)
    assert torch.equal(got_y, y)
    assert all(torch.equal(got_b[n], bal[n]) for n in bal)


def test_binding_refusals_on_the_gpu():
    a, g = _combine_case(16, 64, 4, 2, "bf16")
    with pytest.raises(TypeError):
        M.moe_combine_dropout(**a, residual=torch.zeros(16, 64, device=DEV))
    with pytest.raises(ValueError):
        M.moe_combine_dropout(**dict(a, gate=a["gate"][:8]))
    with pytest.raises(ValueError):
        M.moe_combine_dropout(**dict(a, o=a["o"].t().contiguous().t()))
    with pytest.raises(ValueError):
        M.moe_combine_dropout(**dict(a, rng=a["rng"].cpu()), p=0.5)
    with pytest.raises(M.MoeError):
        M.moe_combine_dropout(**dict(a, rng=None), p=0.5)
    with pytest.raises(M.MoeError):
        M.moe_combine_dropout(**a, p=1.0)
    with pytest.raises(M.MoeError):
        M.moe_combine_dropout(**dict(a, o=torch.zeros(128, 60, device=DEV)))
    b = _route_case(16, 64, 4, 2, "bf16", "softmax_topk", 1.0, True, True, None, False)
    with pytest.raises(M.MoeError):
        M.moe_route_backward(**dict(b, counts=None))
    with pytest.raises(M.MoeError):
        M.moe_route_backward(**dict(b, scores=None))
    with pytest.raises(ValueError):
        M.moe_route_backward(**b, outputs=("dx", "dx"))
    with pytest.raises(M.MoeError):
        M.moe_route_backward(**b, ws=torch.empty(64, dtype=torch.uint8, device=DEV))


def test_the_error_word_is_written_and_clear():
    a = _route_case(*ROUTE[11])
    need = M.moe_route_backward_workspace_bytes(1000, 1024, 8, torch.bfloat16)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    _check_route(a, M.moe_route_backward(**a, ws=ws))
    assert int(ws[:4].view(torch.int32)) == 0


@pytest.mark.parametrize("v", [3.0e38, 3.4e38, -3.4e38, 1e-39, float("inf"), float("nan")])
def test_route_backward_at_the_ends_of_the_range(v):
    """Gate gradients so large, small or not finite that their terms in bf16
    need care: one token, one expert, against the fp64 product."""
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device=DEV)
    x[1, 3] = 1.0
    Wg = torch.zeros((64, 8), dtype=torch.bfloat16, device=DEV)
    Wg[:, 2] = 0.5
    idx = torch.full((4, 1), 2, dtype=torch.int32, device=DEV)
    gate, dgate = torch.zeros((4, 1), device=DEV), torch.zeros((4, 1), device=DEV)
    scores = torch.zeros((8, 4), device=DEV)
    gate[1], dgate[1] = 1.0, v  # softmax over all with p = 0 elsewhere: dz = g dg
    got = M.moe_route_backward(x, Wg, idx, gate, dgate, scores, gating="softmax_topk")
    want = torch.zeros((64, 8), dtype=torch.float64)
    want[3, 2] = v
    dWg, dx = got["dWg"].double().cpu(), got["dx"].double().cpu()
    if v != v or abs(v) == float("inf"):
        assert torch.equal(dWg[3, 2].isnan() | (dWg[3, 2] == v), torch.tensor(True))
        assert bool((dx[1].isnan() | (dx[1] == v)).all())
        return
    # three terms hold v; those below the smallest normal number may be lost
    assert abs(float(dWg[3, 2]) - v) <= 2 * U32 * abs(v) + 2.0 ** -126
    half = torch.full((64,), v / 2, dtype=torch.float64)
    assert torch.all((dx[1] - half).abs() <= (2.0 ** -8 + 2.0 ** -15) * half.abs() + 2.0 ** -126)
    assert not dx[[0, 2, 3]].any()


def test_a_training_step_of_an_empty_batch():
    from mixture_experts_layer_51_b200.workloads import Workload, make_inputs
    w = Workload("t", T=8, d=64, E=4, k=2, H=64, act="swiglu", dtype="bf16", cf=0.0, seed=9)
    t = make_inputs(w, DEV)
    layer = M.MoELayer(t["Wg"], t["bias"], t["W1"], t["W3"], t["W2"], w.k, w.cf, w.act)
    x = t["x"][:0]
    y, loss, step = layer.forward_train(x, coef=0.1)
    assert y.shape == (0, 64) and float(loss) == 0
    layer.backward_combine(step, y)
    grads = layer.backward_router(step)
    assert not grads["dWg"].any() and not grads["dbias"].any() and grads["dx"].shape == (0, 64)


def test_the_step_refuses_what_it_cannot_read():
    from mixture_experts_layer_51_b200.workloads import Workload, make_inputs
    w = Workload("t", T=40, d=64, E=4, k=2, H=64, act="swiglu", dtype="bf16", cf=0.0, seed=9)
    t = make_inputs(w, DEV)
    layer = M.MoELayer(t["Wg"], t["bias"], t["W1"], t["W3"], t["W2"], w.k, w.cf, w.act)
    with pytest.raises(ValueError):
        layer.forward_train(torch.cat([t["x"], t["x"]], 1)[:, :64])
    with pytest.raises(TypeError):
        layer.forward_train(t["x"].float())
    with pytest.raises(M.MoeError):
        layer.forward_train(t["x"], p=0.5)  # no generator
    _, _, step = layer.forward_train(t["x"])
    layer.backward_combine(step, t["x"])
    with pytest.raises(ValueError):
        layer.backward_router(step, dxp=step["xp"][:-128])


@pytest.mark.parametrize("gating,priority,cf,dtype,act", [
    ("topk_softmax", "position", 0.0, "bf16", "swiglu"),
    ("softmax_topk", "position", 1.0, "bf16", "swiglu"),
    ("topk_softmax", "gate", 0.75, "fp32", "gelu")])
def test_a_training_step_of_the_routing(gating, priority, cf, dtype, act):
    """forward_train and the two backward halves, as a training loop calls
    them: every gradient against the oracle on the step's own intermediates,
    and y without dropout and residual against the layer's forward."""
    from mixture_experts_layer_51_b200.workloads import Workload, make_inputs
    w = Workload("t", T=700, d=256, E=8, k=2, H=128, act=act, dtype=dtype, cf=cf, seed=9)
    t = make_inputs(w, DEV)
    layer = M.MoELayer(t["Wg"], t["bias"], t["W1"], t["W3"], t["W2"], w.k, w.cf, w.act,
                       gating=gating, priority=priority)
    x, dt = t["x"], w.torch_dtype
    y0, _, _ = layer.forward_train(x)
    assert torch.equal(y0, layer(x))
    g = _gen(4)
    rng = torch.tensor([42, 7], device=DEV)
    mask = torch.rand(w.T, generator=g, device=DEV) > 0.2
    p = 0.1
    y, loss, step = layer.forward_train(x, coef=0.05, mask=mask, residual=x, p=p, rng=rng)
    keep = oracle.dropout_keep(p, 42, 7, w.T, w.d)
    o, pos, gate = np64(step["o"]), step["pos"].cpu().numpy(), np64(step["gate"])
    want = oracle.combine_dropout(o, pos, gate, keep, p, np64(x))
    size = oracle.combine_dropout(np.abs(o), pos, gate, keep, p)
    assert np.all(np.abs(np64(y) - want) <= 5 * U32 * size + (2 * U32 + _u(dt)) * np.abs(want))
    idx = step["idx"].cpu().numpy()
    want_loss, *_ = oracle.balance_loss(np64(step["scores"]), idx, w.E, 0.05, mask.cpu().numpy())
    assert abs(float(loss) - want_loss) <= w.T * U32 * want_loss
    dy = _randn(g, w.T, w.d, dtype=dt)
    dloss = torch.tensor([300.0], device=DEV)
    d_o = layer.backward_combine(step, dy)
    own = step["pos"][step["pos"] >= 0].long()
    want_o, want_g = oracle.combine_dropout_backward(np64(dy), o, pos, gate, keep, p)
    assert np.all(np.abs(np64(d_o[own]) - want_o[own.cpu().numpy()])
                  <= (3 * U32 + _u(dt)) * np.abs(want_o[own.cpu().numpy()]) + 1e-30)
    # the experts' own gradient of their inputs: anything of that shape
    dxp = _randn(g, *step["xp"].shape, dtype=dt)
    grads = layer.backward_router(step, dloss, dxp)
    acc = M.moe_unpermute_combine(dxp, step["pos"], torch.ones_like(step["gate"]), dt)
    _check_route(dict(x=x, Wg=layer.Wg, idx=step["idx"], scores=step["scores"], mask=mask,
                      gating=gating, gate_scale=1.0, coef=0.05, gate=step["gate"],
                      dgate=step["dgate"], counts=step["balance_counts"], tokens=step["tokens"],
                      dloss=dloss, dx_acc=acc), grads)
    few = layer.backward_router(step, dloss, outputs=("dWg", "dbias"))
    assert torch.equal(few["dWg"], grads["dWg"]) and torch.equal(few["dbias"], grads["dbias"])
