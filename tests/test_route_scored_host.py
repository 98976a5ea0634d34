"""Refusals of routing by scores on the host (nothing reaches the device), and its plain forms."""

import numpy as np
import pytest

from tests import route_scored_ref as ref
from tests.test_abi_host import STATUS, lib  # noqa: F401  (the library fixture)
from tests.test_train_api_host import P, _call


def args(**kw):
    return dict(logits=P, type=0, T=256, E=8, ld=8, bias=None, score=0, groups=2, open=1, best=2, mask=None, k=2,
                renorm=0, scale=1.0, coef=1.0, align=128, max_m=0, ids=P, weights=P, counts=P, routed=P, prob_sum=P,
                loss=P, offsets=P, slots=P, ws=P, ws_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), "SHAPE"), (dict(E=0), "SHAPE"), (dict(k=0), "SHAPE"), (dict(k=5), "SHAPE"), (dict(align=0), "SHAPE"),
    (dict(groups=0), "SHAPE"), (dict(groups=3), "SHAPE"), (dict(open=0), "SHAPE"), (dict(open=3), "SHAPE"),
    (dict(best=0), "SHAPE"), (dict(groups=8, open=2, best=2), "SHAPE"),
    (dict(score=2), "UNSUPPORTED"), (dict(score=-1), "UNSUPPORTED"), (dict(best=3), "UNSUPPORTED"),
    (dict(E=128, ld=128, groups=64, open=8), "UNSUPPORTED"), (dict(type=3), "UNSUPPORTED"),
    (dict(E=1026, ld=1026), "UNSUPPORTED"), (dict(ld=7), "STRIDE"), (dict(logits=None), "NULL"), (dict(slots=None), "NULL"),
    (dict(loss=None), "NULL"), (dict(bias=P + 2), "ALIGN"), (dict(logits=P + 2), "ALIGN"), (dict(ws=P + 8), "ALIGN"),
    (dict(ws_bytes=16), "WORKSPACE"), (dict(ws=None, ws_bytes=0), "WORKSPACE")])
def test_forward(lib, kw, status):  # noqa: F811
    assert _call(lib.moe_route_scored, args(), **kw) == STATUS[status]


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), "SHAPE"), (dict(k=9), "SHAPE"), (dict(score=2), "UNSUPPORTED"), (dict(type=5), "UNSUPPORTED"),
    (dict(ld=7), "STRIDE"), (dict(ldd=7), "STRIDE"), (dict(logits=None), "NULL"), (dict(ids=None), "NULL"),
    (dict(counts=None), "NULL"), (dict(out=None), "NULL"), (dict(dw=P + 2), "ALIGN"), (dict(out=P + 1), "ALIGN"),
    (dict(T=0, logits=None), "OK")])
def test_backward(lib, kw, status):  # noqa: F811
    base = dict(logits=P, type=0, T=256, E=8, ld=8, score=0, ids=P, k=2, renorm=0, scale=1.0, coef=1.0, dw=P, dloss=P,
                counts=P, routed=P, out=P, ldd=8, stream=None)
    assert _call(lib.moe_route_scored_backward, base, **kw) == STATUS[status]


def test_plain_choice_by_hand():
    x = np.array([[0.0, 1.0, 2.0, 3.0, 0.0, 0.0, 9.0, -np.inf]])
    s = ref.scores(x, "sigmoid")
    one = np.ones(1, bool)
    assert ref.select(x, s, None, 1, 1, 1, 3, one).tolist() == [[6, 3, 2]]
    # groups {0,1} {2,3} {4,5} {6,7}: the two best of 2, 3 sum to more than 6 alone
    assert ref.select(x, s, None, 4, 1, 2, 2, one).tolist() == [[3, 2]]
    assert ref.select(x, s, None, 4, 1, 1, 2, one).tolist() == [[6, -1]]
    b = np.zeros(8, np.float32)
    b[0] = 1.0
    assert ref.select(x, s, b, 1, 1, 1, 2, one).tolist() == [[0, 6]]
    # ties: the lower group, the lower expert
    z = np.zeros((1, 8))
    assert ref.select(z, ref.scores(z, "softmax"), None, 4, 2, 1, 3, one).tolist() == [[0, 1, 2]]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [False, True])
def test_plain_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(2)
    T, E, k = 5, 12, 3
    x, dw = rng.standard_normal((T, E)), rng.standard_normal((T, k))
    kw = dict(bias=None, score=score, groups=3, opened=2, best=1, k=k, renorm=renorm, scale=1.7, coef=0.3, align=1, max_m=0)
    o = ref.route(x, **kw)

    def value(y):
        r = ref.route(y, **kw)
        assert np.array_equal(r["expert_ids"], o["expert_ids"])
        return (r["weights"] * dw).sum() + 2.0 * r["loss"]
    got, _ = ref.backward(x, o["expert_ids"], dw, 2.0, o["counts"], o["routed"], score, renorm, 1.7, 0.3)
    h = 1e-5
    for t in range(T):
        for e in range(E):
            d = np.zeros((T, E))
            d[t, e] = h
            assert abs((value(x + d) - value(x - d)) / (2 * h) - got[t, e]) < 1e-8
