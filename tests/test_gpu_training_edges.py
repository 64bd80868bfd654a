"""The training operators where their arithmetic, their waits and their callers
are at an edge: cancelling sums, infinities, time-outs, tensors that autograd
watches, batches split over ranks.

Tolerances are rounding counts, as in test_gpu_training.py: u = 2^-24 is half
a step of fp32, 2^-8 of bf16.  A sum in tensor memory does not round to
nearest: each of its steps is off by at most a whole step, 2 u.
"""

import numpy as np
import pytest
import torch

import oracle
from mixture_experts_layer_51_b200 import moe as M

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
DEV = "cuda"

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
