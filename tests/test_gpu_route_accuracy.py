"""How exact the probabilities are that routing writes out, for experts far
below a row's largest logit."""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_quantizer_amd as fp8g
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu

U = 2.0 ** -24                                  # half a step of fp32, relative
TYPES = {"f32": (torch.float32, 64), "bf16": (torch.bfloat16, 2), "f16": (torch.float16, 16)}


def rows(T, E, t, seed):
    """One logit of 0 in each row, the others 24 to 80 below it and multiples
    of what the type holds there: the differences are exact, and the others' exponentials
    add up to less than 2^-25, so that the sum is 1 in fp32."""
    dtype, per = TYPES[t]
    g = np.random.default_rng(seed)
    x = -g.integers(24 * per, 80 * per + 1, size=(T, E)) / per
    top = g.integers(0, E, size=T)
    x[np.arange(T), top] = 0.0
    v = torch.from_numpy(x).to(dtype)
    assert np.array_equal(v.double().numpy(), x)
    return v.to(dev()), x, top


def routed(x, k, renorm):
    T, E = x.shape
    i, f = torch.int32, torch.float32
    new = lambda s, t: torch.full(s, 77, dtype=t, device=dev())  # noqa: E731
    out = dict(expert_ids=new((T, k), i), weights=new((T, k), f), counts=new((E,), i), routed=new((1,), i),
               prob_sum=new((E,), f), loss=new((1,), f), group_offsets=new((E + 1,), i), slots=new((T, k), i))
    ws = torch.empty(fp8g.moe_route_workspace_size(T, E) + 16, dtype=torch.uint8, device=dev())
    fp8g.moe_route(x, k, *out.values(), ws, renormalise=renorm)
    return out


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,E", [(1, 16), (3, 200), (300, 16), (300, 48), (200, 160), (200, 256), (100, 600)])
def test_weights_of_experts_far_below_the_largest(T, E, t):
    x, exact, _ = rows(T, E, t, T + E)
    for renorm in (False, True):
        out = routed(x, min(E, 16), renorm)
        ids = out["expert_ids"].cpu().numpy()
        want = np.exp(exact[np.arange(T)[:, None], ids])
        off = np.abs(out["weights"].double().cpu().numpy() / want - 1)
        # the exponential instruction's error, one step (2 U), the correction's
        # rounding (U) and the quotient's (U, by a sum of 1); U more for second order
        assert off.max() <= 5 * U, off.max() / U


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,E", [(1, 16), (3, 200), (64, 256), (50, 600)])
def test_sums_of_small_probabilities(T, E, t):
    x, exact, top = rows(T, E, t, T * E)
    out = routed(x, 1, False)
    p = np.exp(exact)
    want = p.sum(0)
    small = ~np.isin(np.arange(E), top)                  # experts that no row has at its top
    off = np.abs(out["prob_sum"].double().cpu().numpy() / want - 1)[small]
    # a probability as above; up to 64 of them added in at most 4 + 2 + 4 roundings
    assert off.max() <= (5 + 10) * U, off.max() / U
