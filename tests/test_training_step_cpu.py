"""The training step's host side, without a GPU: which device its calls run on,
and what its checks of tensors refuse."""

import pytest
import torch

from mixture_experts_layer_51_b200 import moe as M

CALLS = ("moe_route", "moe_expert_choice_route", "moe_balance_loss", "moe_priority_order",
         "moe_permute", "moe_grouped_ffn", "moe_combine_dropout", "moe_combine_dropout_backward",
         "moe_unpermute_combine", "moe_route_backward")


@pytest.fixture
def step(monkeypatch):
    """A layer on the second device of a machine whose first is current; every
    library call notes which device it would have run on."""
    now, seen = [0], []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, now[0] = now[0], self.index

        def __exit__(self, *exc):
            now[0] = self.before

    z = torch.zeros
    results = dict(moe_route=(z(4, 2, dtype=torch.int32), z(4, 2), z(4)),
                   moe_balance_loss=dict(loss=z(1), counts=z(8), tokens=z(1)),
                   moe_permute=dict(xp=z(8, 16), pos=z(4, 2), offsets=z(9), kept_counts=z(8)),
                   moe_grouped_ffn=(z(8, 16), z(8, 16), z(1)),
                   moe_combine_dropout_backward=(z(8, 16), z(4, 2)))

    def fake(name):
        def call(*args, **kwargs):
            seen.append((name, now[0]))
            return results.get(name, z(4, 16))
        return call
    for name in CALLS:
        monkeypatch.setattr(M, name, fake(name))
    monkeypatch.setattr(M, "_current_device", lambda: now[0])
    monkeypatch.setattr(M, "_tensor", lambda *args: 0)
    monkeypatch.setattr(M, "_workspace", lambda *args: z(64, dtype=torch.uint8))
    monkeypatch.setattr(M, "moe_capacity", lambda *args: 4)
    monkeypatch.setattr(torch.cuda, "device", Device)
    layer = M.MoELayer(z(16, 8), None, z(8, 16, 32), z(8, 16, 32), z(8, 32, 16), 2, 1.0,
                       priority="gate")
    layer.device = torch.device("cuda", 1)
    return layer, now, seen


def test_every_call_of_a_step_runs_on_the_layer_device(step):
    layer, now, seen = step
    y, _, s = layer.forward_train(torch.zeros(4, 16), coef=0.1)
    layer.backward_combine(s, y)
    layer.backward_router(s, dxp=torch.zeros(8, 16))
    assert {name for name, _ in seen} == set(CALLS)
    assert all(device == 1 for _, device in seen), seen
    assert now[0] == 0
    now[0] = 1  # already current: nothing to switch
    layer.backward_combine(s, y)
    assert seen[-1] == ("moe_combine_dropout_backward", 1) and now[0] == 1


def test_the_device_is_put_back_after_an_error(step, monkeypatch):
    layer, now, _ = step

    def refuse(*args, **kwargs):
        raise M.MoeError(M.MOE_ERR_ARG, "moe_permute")
    monkeypatch.setattr(M, "moe_permute", refuse)
    with pytest.raises(M.MoeError):
        layer.forward_train(torch.zeros(4, 16))
    assert now[0] == 0


def test_a_tensor_that_autograd_watches_is_refused():
    """... and passes where autograd does not record."""
    w = torch.zeros(3, requires_grad=True)
    with pytest.raises(ValueError, match="t requires a gradient"):
        M._tensor(w, "t", torch.float32, (3,), -1)
    with pytest.raises(ValueError, match="t requires a gradient"):
        M._tensor(w * 2, "t", torch.float32, (3,), -1)
    assert M._tensor(w.detach(), "t", torch.float32, (3,), -1) == w.data_ptr()
    with torch.no_grad():
        assert M._tensor(w, "t", torch.float32, (3,), -1) == w.data_ptr()


@pytest.mark.parametrize("name", ["Wg", "W1", "W3", "W2"])
def test_the_step_refuses_weights_that_autograd_watches(step, name):
    layer, _, seen = step
    setattr(layer, name, torch.nn.Parameter(getattr(layer, name)))
    with pytest.raises(ValueError, match=f"{name} requires a gradient"):
        layer.forward_train(torch.zeros(4, 16))
    assert not seen
    with torch.no_grad():
        layer.forward_train(torch.zeros(4, 16))
    assert seen


def test_a_tensor_that_is_not_dense_is_refused():
    """By its strides: type, shape and device (-1: not on a GPU) are right."""
    t = torch.zeros(4, 3).t()
    with pytest.raises(ValueError, match="t is not contiguous"):
        M._tensor(t, "t", torch.float32, (3, 4), -1)
    assert M._tensor(t.contiguous(), "t", torch.float32, (3, 4), -1) is not None
    with pytest.raises(ValueError, match="t is on cpu, expected cuda:0"):
        M._tensor(t, "t", torch.float32, (3, 4), 0)
