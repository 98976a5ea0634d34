"""The operators together: the example layer's gradients against torch's
differentiation of the same layer, and its training."""

import pytest
import torch

from examples.moe_train_step import MoELayer, train
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu


def _reference(layer, x, dy, mask):
    """Loss gradients in fp64 with the layer's own choice of experts."""
    W = layer.weight.double().requires_grad_(True)
    router = layer.router.double().requires_grad_(True)
    ids = layer.route["expert_ids"].long()
    live = ids >= 0
    on = live[:, 0]
    p = torch.softmax(x.double() @ router.t(), 1)
    w = torch.where(live, p.gather(1, ids.clamp(min=0)), torch.zeros((), dtype=p.dtype, device=p.device))
    w = w / torch.where(on, w.sum(1), torch.ones_like(w[:, 0]))[:, None]
    y = torch.zeros(x.shape[0], layer.N, dtype=torch.float64, device=x.device)
    for e in range(layer.E):
        share = torch.where(ids == e, w, torch.zeros_like(w)).sum(1)
        y = y + share[:, None] * (x.double() @ W[e].t())
    n = on.sum().double()
    counts = torch.bincount(ids[live], minlength=layer.E).double()
    balance = layer.balance * (layer.E * counts / (layer.k * n) * p[on].sum(0) / n).sum()
    ((y * dy.double()).sum() + balance).backward()
    return y.detach(), W.grad, router.grad, balance.detach()


def _off(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("masked", [False, True])
def test_gradients_against_torch(masked):
    torch.manual_seed(0)
    layer = MoELayer(700, 256, 384, 6, 2, seed=3)
    x = torch.randn(700, 256, device=dev()).to(torch.bfloat16)
    mask = torch.rand(700, device=dev()) > 0.3 if masked else None
    y = layer.forward(x, mask)
    dy = torch.randn(700, 384, device=dev()) * 1e-2
    if masked:
        dy = dy * mask[:, None]
        assert (y[~mask] == 0).all()
    dW, dR = layer.backward(x, dy)
    ry, rW, rR, balance = _reference(layer, x, dy, mask)
    # each 8-bit rounding is off by at most 2^-4 (e4m3) or 2^-3 (e5m2) of its
    # value, evenly spread over half that and averaged over independent terms: the norm
    # of the sum is off by less than the quadratic sum of the two maxima / sqrt(3)
    assert _off(y, ry) < (2 * 2.0 ** -8) ** 0.5 / 3 ** 0.5
    assert _off(dW, rW) < (2.0 ** -8 + 2.0 ** -6) ** 0.5 / 3 ** 0.5
    # the router's gradient goes by the forward product's values
    assert _off(dR, rR) < 2 * (2 * 2.0 ** -8) ** 0.5 / 3 ** 0.5
    # (the logits are fp32 products of 256 terms)
    assert abs(float(layer.route["loss"]) - float(balance)) < 1e-5 * float(balance)


def test_it_trains():
    losses = train(steps=25)
    assert all(v == v for v in losses)
    assert losses[-1] < 0.5 * losses[0], losses
