"""Routing by scores on the GPU where its documentation allows what the other tests do not do."""

import numpy as np
import pytest
import torch

from tests.gpu_util import dev
from tests.test_gpu_route_scored import TYPES, check, logits, some_bias

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,groups", [(3, 256, 1), (70, 16, 2), (70, 60, 5), (70, 128, 1), (70, 192, 12), (70, 256, 8),
                                        (40, 512, 16), (20, 1024, 32)])
def test_closed_experts_are_never_chosen(T, E, groups, score, kind):
    """Closed by a bias of -inf or NaN, by a logit of -inf or (for a token that is not in the sums) a mask, half
    of them and more; experts past the last, in a lane's registers, are closed as well."""
    rng = np.random.default_rng(E + T)
    x = logits(rng, T, E, kind)
    shut = rng.permutation(E)
    x[:, torch.from_numpy(shut[:E // 4]).to(dev())] = -torch.inf
    bias = some_bias(rng, E)
    bias[shut[E // 4:E // 2]] = -np.inf
    bias[shut[E // 2:5 * E // 8]] = np.nan
    mask = rng.random(T) > 0.2
    k = min(8, E // groups)
    for b in (bias, None):
        for opened in {groups, max(1, groups // 2)}:
            got = check(x, k, b, score, groups, opened, min(2, E // groups), mask, True, 2.5)
            never = shut[:E // 4] if b is None else shut[:5 * E // 8]
            assert not np.isin(got["expert_ids"], never).any()
            assert (got["expert_ids"][~mask] == -1).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,groups,k", [(16, 1, 4), (64, 8, 6), (192, 12, 8), (256, 1, 8), (256, 8, 8), (512, 16, 8),
                                        (1024, 1, 16), (1024, 32, 8)])
@pytest.mark.parametrize("size", [0.25, 0.5, 1.0, 2.0])
def test_near_values_of_scores_that_differ(E, groups, k, score, size):
    """Biases about as large as the largest score (`size` of it) that make up for the scores' differences: what
    all scores of a row share of their error does not cancel between two values then."""
    rng = np.random.default_rng(E + int(size * 8))
    x = (rng.standard_normal((90, E)) * 2).astype(np.float32)
    top = np.float32(3.0)
    near = rng.permutation(E)[:max(k + 4, E // 2)]     # (others lie below, a few of them far)
    x[:, near[0]] = top + 3
    base = np.exp(x[0].astype(np.float64) - x[0].max())
    s = 1 / (1 + np.exp(-x[0].astype(np.float64))) if score == "sigmoid" else base / base.sum()
    bias = (size * s.max() - s).astype(np.float32)
    bias[np.setdiff1d(np.arange(E), near)] -= np.float32(s.max() / 4)
    x[1::2] = x[0]
    # rows like the first but for steps of a few 2^-22 of a logit
    x[1::2] *= (1 + rng.integers(-3, 4, x[1::2].shape) * 2.0 ** -23).astype(np.float32)
    x[2::4] = x[0] + np.float32(0.5)                   # (softmax: the same scores, rounded otherwise)
    check(torch.from_numpy(x).to(dev()), k, bias, score, groups, max(1, groups // 2), min(2, E // groups))
