"""The many-row reference of routing against the oracle."""

import numpy as np
import pytest

from oracle import train
from tests import route_ref


@pytest.mark.parametrize("renorm,max_m,align", [(False, 0, 128), (True, 0, 1), (True, 7, 128)])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (90, 13, 4), (200, 40, 16)])
def test_against_the_oracle(T, E, k, renorm, max_m, align):
    g = np.random.default_rng(T + E)
    x = np.round(g.normal(size=(T, E)) * 4) / 2
    if T > 1:
        x[:, ::5] = -np.inf
        x[::9] = -np.inf
        x[1::9, 2:] = -np.inf
    mask = g.random(T) > 0.2 if T > 1 else None
    kw = dict(mask=mask, renormalise=renorm, coef=0.3, align=align, max_m=max_m)
    a, b = route_ref.route(x, k, **kw), train.route(x, k, **kw)
    for n in a:
        if np.asarray(b[n]).dtype.kind == "f":
            np.testing.assert_allclose(a[n], b[n], rtol=1e-12, atol=1e-300, err_msg=n)
        else:
            assert np.array_equal(a[n], b[n]), n
    dw = g.normal(size=(T, k))
    args = (x, b["expert_ids"], dw, 1.7, b["counts"], b["routed"], renorm, 0.3)
    for u, v in zip(route_ref.route_backward(*args), train.route_backward(*args)):
        np.testing.assert_allclose(u, v, rtol=1e-11, atol=1e-14)
