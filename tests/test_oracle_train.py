"""The training-step oracle against facts that do not come from it:
differences of its own forward for the gradients, torch's differentiation and
casts, exact rationals for the scales."""

from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import train
from oracle.formats import FORMATS


def _objective(x, k, dw, dl, renorm, coef, ids, mask):
    """sum(weights * dw) + dl * loss, with the choice held fixed."""
    p = train.softmax(x)
    total = 0.0
    for t in range(x.shape[0]):
        live = [j for j in range(k) if ids[t, j] >= 0]
        w = p[t, ids[t, live]]
        if renorm and live:
            w = w / w.sum()
        total += float((w * dw[t, live]).sum())
    on = ids[:, 0] >= 0
    n = max(int(on.sum()), 1)
    counts = np.bincount(ids[ids >= 0], minlength=x.shape[1])
    return total + dl * coef * float((x.shape[1] * counts / (k * n) * p[on].sum(0) / n).sum())


@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_against_differences(renorm):
    rng = np.random.default_rng(3)
    T, E, k = 7, 6, 3
    x = rng.normal(size=(T, E))
    x[2, 1] = x[5, 3] = -np.inf
    x[6, 2:] = -np.inf                                     # fewer experts than k
    mask = np.array([1, 1, 1, 0, 1, 1, 1], bool)
    r = train.route(x, k, mask=mask, renormalise=renorm, coef=0.3)
    dw, dl = rng.normal(size=(T, k)), 1.7
    g, _ = train.route_backward(x, r["expert_ids"], dw, dl, r["counts"], r["routed"], renorm, 0.3)
    h = 1e-6
    for t in range(T):
        for e in range(E):
            if x[t, e] == -np.inf:
                assert g[t, e] == 0
                continue
            up, dn = x.copy(), x.copy()
            up[t, e] += h
            dn[t, e] -= h
            args = (k, dw, dl, renorm, 0.3, r["expert_ids"], mask)
            d = (_objective(up, *args) - _objective(dn, *args)) / (2 * h)
            # central differences in float64: h^2 of the third derivative
            # (below 10 here) and 2^-52 / h of the values (below 10)
            assert abs(d - g[t, e]) < 1e-8, (t, e)


def test_gradient_against_torch():
    rng = np.random.default_rng(4)
    x = rng.normal(size=(40, 12))
    r = train.route(x, 4, renormalise=True, coef=0.02)
    dw = rng.normal(size=(40, 4))
    xt = torch.tensor(x, requires_grad=True)
    p = torch.softmax(xt, 1)
    w = p.gather(1, torch.tensor(r["expert_ids"]).long())
    w = w / w.sum(1, keepdim=True)
    f = 12 * torch.tensor(r["counts"]).double() / (4 * 40)
    loss = 0.02 * (f * p.mean(0)).sum()
    assert abs(float(loss) - r["loss"]) < 1e-14
    np.testing.assert_allclose(w.detach().numpy(), r["weights"], rtol=1e-13)
    ((w * torch.tensor(dw)).sum() + 3.0 * loss).backward()
    g, _ = train.route_backward(x, r["expert_ids"], dw, 3.0, r["counts"], r["routed"], True, 0.02)
    np.testing.assert_allclose(g, xt.grad.numpy(), atol=1e-14)


def test_choice_ties_masks_and_slots():
    inf, nan = np.inf, np.nan
    x = np.array([[1.0, 2.0, 2.0, 0.0], [-inf, -inf, -inf, -inf], [0.0, -0.0, 0.0, -inf],
                  [nan, 1.0, -inf, -inf], [3.0, 3.0, 3.0, 3.0]])
    r = train.route(x, 2, mask=[1, 1, 1, 1, 0], align=4)
    assert r["expert_ids"].tolist() == [[1, 2], [-1, -1], [0, 1], [1, -1], [-1, -1]]
    assert np.isnan(r["weights"][3]).all() and np.isnan(r["loss"])
    assert (r["weights"][[1, 4]] == 0).all()
    assert r["counts"].tolist() == [1, 3, 1, 0] and r["routed"] == 3
    assert r["group_offsets"].tolist() == [0, 4, 8, 12, 12]
    assert r["slots"].tolist() == [[4, 8], [-1, -1], [0, 5], [6, -1], [-1, -1]]
    r = train.route(x[[0, 2, 2]], 2, max_m=2)
    assert r["group_offsets"].tolist() == [0, 2, 4, 6, 8]
    assert r["slots"].tolist() == [[2, 4], [0, 3], [1, -1]] and r["counts"].tolist() == [2, 3, 1, 0]


def test_an_even_routing_has_the_loss_coef():
    x = np.zeros((8, 4))
    for t in range(8):
        x[t, t % 4] = 50.0
    assert abs(train.route(x, 1, coef=0.7)["loss"] - 0.7) < 1e-12


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_scales_are_the_smallest_powers_and_codes_are_nearest(fmt):
    rng = np.random.default_rng(5)
    top = FORMATS[fmt][0]
    x = (rng.normal(size=(300, 24)) * 10.0 ** rng.uniform(-6, 6, size=(1, 24))).astype(np.float32)
    x[128:256, 3] = 0
    for j, v in enumerate((top, np.nextafter(np.float32(top), np.float32(1e9)), top * 2.0 ** -20)):
        x[:128, 4 + j] = 0
        x[7, 4 + j] = v
    q, s = train.quantize_transpose(x, fmt)
    assert q.shape == (24, 384) and s.shape == (3, 24) and (q[:, 300:] == 0).all()
    for i in range(3):
        for c in range(24):
            amax = Fraction(float(np.abs(x[i * 128:(i + 1) * 128, c]).max()))
            e = int(s[i, c]) - 127
            if amax == 0:
                assert e == 0
                continue
            assert amax <= Fraction(top) * Fraction(2) ** e
            assert amax > Fraction(top) * Fraction(2) ** (e - 1)
    t = torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2
    want = (x / np.ldexp(np.float32(1), np.repeat(s.astype(int) - 127, 128, axis=0)[:300])).astype(np.float32)
    want = torch.from_numpy(want).to(t).view(torch.uint8).numpy()
    assert np.array_equal(q[:, :300], want.T)


def test_wgrad_of_small_integers_is_an_integer_product():
    rng = np.random.default_rng(6)
    a = rng.integers(-8, 9, size=(300, 16)).astype(np.float32)
    b = rng.integers(-8, 9, size=(300, 32)).astype(np.float32)
    qa, sa = train.quantize_transpose(a, "e4m3")
    qb, sb = train.quantize_transpose(b, "e4m3")
    d, _ = train.wgrad(qa, "e4m3", sa, qb, "e4m3", sb, [0, 128, 128, 384])
    assert np.array_equal(d[0], a[:128].T @ b[:128])
    assert (d[1] == 0).all()
    assert np.array_equal(d[2], a[128:].T @ b[128:])


def test_clip():
    total, norm, out = train.grad_clip([np.array([3.0]), np.array([]), np.array([4.0])], 1.0)
    assert total == 25 and norm == 5 and abs(out[0][0] - 0.6) < 1e-6 and out[1].size == 0
    assert train.grad_clip([np.array([0.3])], 1.0)[2][0][0] == 0.3
