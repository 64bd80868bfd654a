"""CPU checks of the training entry points: argument checks of the C ABI and
of the binding happen before anything is enqueued (no GPU)."""

import ctypes
import math

import pytest
import torch

from mixture_experts_layer_51_b200 import moe as M

F = ctypes.c_void_p(0x10000)     # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10002)   # not aligned to a float
HALF = ctypes.c_void_p(0x10008)  # aligned to 8, not to 16
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return M.lib()


def _balance(lib, **kw):
    a = dict(scores=F, idx=F, mask=None, T=100, E=8, k=2, coef=0.01, loss=F, prob_sum=F, counts=F,
             tokens=F, ws=F, ws_bytes=BIG, stream=None)
    a.update(kw)
    return lib.moe_balance_loss(*a.values())


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(E=0), dict(E=65), dict(k=0), dict(k=9), dict(E=2, k=3),
    dict(coef=math.nan), dict(coef=math.inf), dict(T=1 << 30, k=2), dict(scores=None),
    dict(idx=None), dict(loss=None), dict(prob_sum=None), dict(counts=None), dict(tokens=None),
    dict(ws=None), dict(ws=HALF), dict(ws_bytes=16), dict(scores=ODD), dict(idx=ODD),
    dict(loss=ODD), dict(prob_sum=ODD), dict(counts=ODD), dict(tokens=ODD)])
def test_balance_loss_refuses(lib, bad):
    assert _balance(lib, **bad) == M.MOE_ERR_ARG


def _route_back(lib, **kw):
    a = dict(x=F, Wg=F, scores=F, idx=F, gate=F, dgate=F, counts=F, tokens=F, dloss=F, coef=0.01,
             mask=None, dx_acc=F, T=100, d=64, E=8, k=2, dtype=M.MOE_BF16, opt=None, dx=F, dWg=F,
             dbias=F, ws=F, ws_bytes=BIG, stream=None)
    a.update(kw)
    return lib.moe_route_backward(*a.values())


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(d=0), dict(d=60), dict(E=65), dict(k=9), dict(E=2, k=3), dict(dtype=7),
    dict(coef=math.nan), dict(dx=None, dWg=None, dbias=None), dict(dx=HALF), dict(dWg=HALF),
    dict(dbias=ODD), dict(dgate=None, counts=None, tokens=None), dict(counts=None),
    dict(tokens=None), dict(counts=ODD), dict(tokens=ODD), dict(dloss=ODD), dict(idx=None),
    dict(gate=None), dict(idx=ODD), dict(gate=ODD), dict(dgate=ODD), dict(scores=None),
    dict(scores=ODD), dict(Wg=None), dict(Wg=HALF), dict(dx_acc=HALF), dict(x=None), dict(x=HALF),
    dict(ws=None), dict(ws=HALF), dict(ws_bytes=16), dict(T=2**31 - 127)])
def test_route_backward_refuses(lib, bad):
    assert _route_back(lib, **bad) == M.MOE_ERR_ARG


@pytest.mark.parametrize("fine", [
    dict(x=None, dWg=None), dict(Wg=None, dx=None), dict(dgate=None, gate=None, idx=None),
    dict(counts=None, tokens=None, scores=None, dloss=None), dict(dloss=None), dict(dx_acc=None),
    dict(dx_acc=HALF, dx=None)])
def test_route_backward_takes_what_it_does_not_need_as_null(lib, fine):
    """Past the checks, to the first CUDA call, which fails without a GPU."""
    if torch.cuda.is_available():
        pytest.skip("would launch on made-up addresses")
    assert _route_back(lib, **fine) not in (M.MOE_OK, M.MOE_ERR_ARG)


def test_route_backward_needs_scores_for_the_switch_order(lib):
    opt = M.moe_options(gating=M.MOE_GATE_SOFTMAX_TOPK, gate_scale=1.0)
    assert _route_back(lib, counts=None, tokens=None, scores=None,
                       opt=ctypes.byref(opt)) == M.MOE_ERR_ARG
    for o in (M.moe_options(gating=3, gate_scale=1.0), M.moe_options(gating=0, gate_scale=0.0)):
        assert _route_back(lib, opt=ctypes.byref(o)) == M.MOE_ERR_ARG


def _combine(lib, **kw):
    a = dict(o=F, pos=F, gate=F, residual=F, p=0.1, rng=F, T=100, d=64, k=2, dtype=M.MOE_BF16, y=F,
             stream=None)
    a.update(kw)
    return lib.moe_combine_dropout(*a.values())


def _combine_back(lib, **kw):
    a = dict(dy=F, o=F, pos=F, gate=F, p=0.1, rng=F, T=100, d=64, k=2, dtype=M.MOE_BF16, d_o=F,
             dgate=F, stream=None)
    a.update(kw)
    return lib.moe_combine_dropout_backward(*a.values())


SIZES = [dict(T=-1), dict(d=0), dict(d=12), dict(k=0), dict(k=9), dict(dtype=5), dict(p=-0.1),
         dict(p=1.0), dict(p=math.nan), dict(rng=None), dict(rng=ctypes.c_void_p(0x10004)),
         dict(o=None), dict(pos=None), dict(gate=None), dict(o=HALF), dict(pos=ODD),
         dict(gate=ODD)]


@pytest.mark.parametrize("bad", SIZES + [dict(y=None), dict(y=HALF), dict(residual=HALF)])
def test_combine_dropout_refuses(lib, bad):
    assert _combine(lib, **bad) == M.MOE_ERR_ARG


@pytest.mark.parametrize("bad", SIZES + [dict(dy=None), dict(dy=HALF), dict(d_o=None),
                                         dict(d_o=HALF), dict(dgate=None), dict(dgate=ODD)])
def test_combine_dropout_backward_refuses(lib, bad):
    assert _combine_back(lib, **bad) == M.MOE_ERR_ARG


def test_empty_batches_are_no_ops(lib):
    assert _combine(lib, T=0, o=None, y=None) == M.MOE_OK
    assert _combine_back(lib, T=0, o=None, dy=None) == M.MOE_OK
    # the loss of an empty batch is written (zeros), so its outputs are needed
    assert _balance(lib, T=0, loss=None) == M.MOE_ERR_ARG


def test_workspace_sizes(lib):
    assert M.moe_balance_loss_workspace_bytes(-1, 8) == 0
    assert M.moe_balance_loss_workspace_bytes(10, 65) == 0
    assert 0 < M.moe_balance_loss_workspace_bytes(0, 8) <= M.moe_balance_loss_workspace_bytes(
        100000, 8)
    assert M.moe_route_backward_workspace_bytes(10, 12, 8, torch.bfloat16) == 0
    assert M.moe_route_backward_workspace_bytes(10, 64, 65, torch.bfloat16) == 0
    # the end of the last tile of tokens is an int32 too
    assert M.moe_route_backward_workspace_bytes(2**31 - 127, 64, 8, torch.float32) == 0
    assert M.moe_route_backward_workspace_bytes(2**31 - 128, 64, 8, torch.float32) >= 2**31 * 4
    for dt in (torch.bfloat16, torch.float32):
        # room for dz at least, and bounded by a few copies of dz and dWg
        need = M.moe_route_backward_workspace_bytes(10000, 2048, 64, dt)
        assert 10000 * 64 * 4 <= need <= 64 << 20


def test_binding_refuses_what_a_pointer_cannot_carry():
    """CPU tensors, wrong types, shapes and strides never reach the library."""
    z = torch.zeros
    with pytest.raises(ValueError):
        M.moe_balance_loss(z(8, 10), z(10, 2, dtype=torch.int32), 0.01)
    with pytest.raises(ValueError):
        M.moe_combine_dropout(z(128, 64), z(4, 2, dtype=torch.int32), z(4, 2))
    with pytest.raises(ValueError):
        M.moe_combine_dropout_backward(z(4, 64), z(128, 64), z(4, 2, dtype=torch.int32), z(4, 2))
    with pytest.raises(ValueError):
        M.moe_route_backward(z(4, 64), z(64, 8), z(4, 2, dtype=torch.int32), z(4, 2), z(4, 2))
    cpu = torch.device("cpu")
    with pytest.raises(TypeError):
        M._tensor(z(3), "t", torch.int32, (3,), cpu)
    with pytest.raises(ValueError):
        M._tensor(z(3), "t", torch.float32, (4,), cpu)
    with pytest.raises(ValueError):
        M._tensor(z(4, 3).t(), "t", torch.float32, (3, 4), cpu)
    with pytest.raises(ValueError):
        M._tensor(z(3), "t", torch.float32, (3,), torch.device("cuda", 0))
    assert M._tensor(None, "t", torch.float32, (3,), cpu) is None
