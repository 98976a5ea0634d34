"""Scored routing, products in 8-bit integers and the AdamW step together, as the example's
layer uses them: its gradients against torch's differentiation, its answers against the exact
layer, its updates against the definition."""

import numpy as np
import pytest
import torch

from examples.moe_train_step import MoELayer
from tests import adamw_ref
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu

OPTIONS = [dict(score="sigmoid"), dict(score="softmax"), dict(score="sigmoid", groups=4, open_groups=2)]


def _exact(layer, x, W, router):
    """fp64 y, shares and balance loss, by the layer's own choice of experts."""
    ids = layer.route["expert_ids"].long()
    live = ids >= 0
    on = live[:, 0]
    z = x.double() @ router.t()
    s = torch.sigmoid(z) if layer.scored["score"] == "sigmoid" else torch.softmax(z, 1)
    w = torch.where(live, s.gather(1, ids.clamp(min=0)), torch.zeros((), dtype=s.dtype, device=s.device))
    w = w / torch.where(on, w.sum(1), torch.ones_like(w[:, 0]))[:, None]
    y = torch.zeros(x.shape[0], layer.N, dtype=torch.float64, device=x.device)
    for e in range(layer.E):
        share = torch.where(ids == e, w, torch.zeros_like(w)).sum(1)
        y = y + share[:, None] * (x.double() @ W[e].t())
    n = on.sum().double()
    counts = torch.bincount(ids[live], minlength=layer.E).double()
    p = s[on] / s[on].sum(1, keepdim=True)
    balance = layer.balance * (layer.E * counts / (layer.k * n) * p.sum(0) / n).sum()
    return y, balance


def _off(a, b):
    return float((a.double() - b).norm() / b.norm())


def _problem(options, masked, **more):
    torch.manual_seed(0)
    layer = MoELayer(700, 256, 384, 8, 2, seed=3, **options, **more)
    layer.bias.copy_(torch.linspace(-0.1, 0.1, 8))
    x = torch.randn(700, 256, device=dev()).to(torch.bfloat16)
    return layer, x, torch.rand(700, device=dev()) > 0.3 if masked else None


@pytest.mark.parametrize("options", OPTIONS)
@pytest.mark.parametrize("masked", [False, True])
def test_gradients_against_torch(options, masked):
    layer, x, mask = _problem(options, masked)
    y = layer.forward(x, mask)
    dy = torch.randn(700, 384, device=dev()) * 1e-2
    if masked:
        dy = dy * mask[:, None]
        assert (y[~mask] == 0).all()
    dW, dR = layer.backward(x, dy)
    W = layer.weight.double().requires_grad_(True)
    router = layer.router.double().requires_grad_(True)
    ry, balance = _exact(layer, x, W, router)
    ((ry * dy.double()).sum() + balance).backward()
    # each 8-bit rounding is off by at most 2^-4 (e4m3) or 2^-3 (e5m2) of its value, evenly spread
    # over half that and averaged over independent terms: the norm of the sum is off by less than
    # the quadratic sum of the two maxima / sqrt(3)
    assert _off(y, ry.detach()) < (2 * 2.0 ** -8) ** 0.5 / 3 ** 0.5
    assert _off(dW, W.grad) < (2.0 ** -8 + 2.0 ** -6) ** 0.5 / 3 ** 0.5
    # the router's gradient goes by the forward product's values
    assert _off(dR, router.grad) < 2 * (2 * 2.0 ** -8) ** 0.5 / 3 ** 0.5
    # (the logits are fp32 products of 256 terms)
    assert abs(float(layer.route["loss"]) - float(balance.detach())) < 1e-5 * float(balance.detach())


@pytest.mark.parametrize("options", OPTIONS)
@pytest.mark.parametrize("masked", [False, True])
def test_served_answers(options, masked):
    layer, x, mask = _problem(options, masked)
    layer.freeze()
    y = layer.serve(x, mask)
    ry, _ = _exact(layer, x, layer.weight.double(), layer.router.double())
    # an operand's rounding is off by at most half a step, amax / 254 of the row, independently and
    # evenly spread (1 / sqrt(3) of that in the mean): against the row's mean square; and the bf16
    # result's, 2^-8
    step = [float((m.double().abs().amax(-1) / 254 / m.double().square().mean(-1).sqrt()).max())
            for m in (x, layer.weight)]
    assert _off(y, ry) < (sum(v * v for v in step) / 3 + 2.0 ** -16) ** 0.5
    if masked:
        assert (y[~mask] == 0).all()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("max_norm", [0.5, 0.01])      # (above the gradients' norm, and below it)
def test_updates_by_the_definition(bits, max_norm):
    """Three steps: the layer's weights after each, from its own gradients and states."""
    layer, x, _ = _problem(OPTIONS[2], False, adamw=bits)
    target = torch.randn(700, 384, device=dev())
    lr, b1, b2, eps, decay = 3e-3, 0.9, 0.999, 1e-8, 0.01
    params = [layer.weight, layer.router]
    host = lambda t: t.detach().cpu().numpy().reshape(-1)  # noqa: E731
    bias = layer.bias.clone()
    for step in (1, 2, 3):
        before, states = [host(p).copy() for p in params], [[host(t).copy() for t in s] for s in layer.states]
        layer.step(x, target, lr, max_norm=max_norm)
        sumsq = float(layer.sumsq)
        grads = [host(g.float()) for g in (layer.d_weight, layer.d_router)]
        total = sum(float((g.astype(np.float64) ** 2).sum()) for g in grads)
        assert abs(sumsq - total) < 2.0 ** -22 * total and 0.01 < sumsq ** 0.5 < 0.5
        clip = adamw_ref.factor(sumsq, max_norm)
        for i, (p, old, g) in enumerate(zip(params, before, grads)):
            if bits == 32:
                m, v = states[0][i], states[1][i]
            else:
                m, r = [adamw_ref.decode(states[k][i], states[k + 2][i]).astype(np.float32) for k in (0, 1)]
                v = r * r
            m, v, r = adamw_ref.states(g, m, v, clip, b1, b2)
            if bits == 32:
                assert np.array_equal(host(layer.states[0][i]), m) and np.array_equal(host(layer.states[1][i]), v)
            want, u = adamw_ref.params(old, m, r, step, lr, b1, b2, eps, decay)
            # p (1 - lr wd): the factor's and the product's rounding; the update: size, inv, r inv,
            # + eps, the reciprocal (two half steps), two products; their difference; fp32's
            tol = 2.0 ** -24 * (np.abs(want) * 4 + u * 10) + 2.0 ** -149
            assert (np.abs(host(p) - want) <= tol).all()
    assert (layer.bias != bias).any()


def test_a_step_that_overflowed_changes_nothing():
    layer, x, _ = _problem(OPTIONS[0], False, adamw=32)
    target = torch.randn(700, 384, device=dev())
    target[5, 7] = float("inf")
    before = [p.clone() for p in (layer.weight, layer.router, *layer.states[0], *layer.states[1])]
    layer.step(x, target, 3e-3)
    assert not torch.isfinite(layer.sumsq).all()
    assert all(torch.equal(a, b) for a, b in zip(before, (layer.weight, layer.router, *layer.states[0],
                                                          *layer.states[1])))
